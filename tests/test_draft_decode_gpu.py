"""The drafted-decode example against a plain 64-bit forward pass without caches, states or drafts: greedy runs give the
model's own greedy tokens, sampled ones follow from the random numbers and the model's probabilities."""
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
    spec = importlib.util.spec_from_file_location("draft_decode", os.path.join(ROOT, "examples", "draft_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.qg.load()
    m.qg.device_status()
    return m


class Plain:
    """The same decoder in 64 bits from dequantized weights; q, k and v of attention round to f16 as the cache does."""

    def __init__(self, w, c, oracle, gs):
        d = lambda b, r, n: torch.from_numpy(oracle.dequant(gs.Q8_0, b.reshape(-1), r, n)).double()  # noqa: E731
        f = lambda a: torch.from_numpy(a).double()  # noqa: E731
        self.c, self.embed, self.final = c, d(w.embed, c.V, c.H), f(w.final)
        self.delta = [d(x, m, c.H) for x, m in zip(w.delta, (c.Hk * c.Dk, c.Hk * c.Dk, c.Hv * c.Dv))]
        self.gates = [d(x, c.Hv, c.H) for x in w.gates]
        self.delta_out, self.attn_out = d(w.delta_out, c.H, c.Hv * c.Dv), d(w.attn_out, c.H, c.Hq * c.D)
        self.attn = [d(x, m, c.H) for x, m in zip(w.attn, (c.Hq * c.D, c.Hkv * c.D, c.Hkv * c.D))]
        self.a_scale, self.a_bias = f(w.a_scale), f(w.a_bias)

    def norm(self, x, w=1.0):
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + self.c.eps) * w

    def rope(self, x):
        h = self.c.D // 2
        f = self.c.theta ** (-2.0 * torch.arange(h, dtype=torch.float64) / self.c.D)
        a = torch.arange(x.shape[0], dtype=torch.float64)[:, None, None] * f
        u, v = x[..., :h], x[..., h:]
        return torch.cat([u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos()], -1)

    def logits(self, tokens):
        c, n = self.c, len(tokens)
        x = self.embed[torch.as_tensor(tokens, dtype=torch.long)]
        xn = self.norm(x)
        q, k = [(xn @ m.T).view(n, c.Hk, c.Dk) for m in self.delta[:2]]
        v = (xn @ self.delta[2].T).view(n, c.Hv, c.Dv)
        q, k = [(t / torch.sqrt(t.square().sum(-1, keepdim=True) + c.eps)).repeat_interleave(c.Hv // c.Hk, 1) for t in (q, k)]
        alpha = torch.exp(self.a_scale * torch.nn.functional.softplus(xn @ self.gates[0].T + self.a_bias))
        beta = torch.sigmoid(xn @ self.gates[1].T)
        S, o = torch.zeros(c.Hv, c.Dk, c.Dv, dtype=torch.float64), []
        for t in range(n):
            S = alpha[t, :, None, None] * S
            S = S + k[t, ..., None] * (beta[t, :, None] * (v[t] - torch.einsum("hij,hi->hj", S, k[t])))[:, None]
            o.append(torch.einsum("hij,hi->hj", S, q[t]) * c.Dk ** -0.5)
        x = x + c.mix * (torch.stack(o).reshape(n, -1) @ self.delta_out.T)
        xn = self.norm(x)
        r16 = lambda t: t.float().half().double()  # noqa: E731
        q, k, v = [(xn @ m.T).view(n, -1, c.D) for m in self.attn]
        q, k, v = r16(self.rope(self.norm(q))), r16(self.rope(self.norm(k))), r16(v)
        g = c.Hq // c.Hkv
        s = torch.einsum("thd,shd->hts", q, k.repeat_interleave(g, 1)) / math.sqrt(c.D)
        s = s.masked_fill(torch.triu(torch.ones(n, n, dtype=torch.bool), 1), -math.inf)
        x = x + c.mix * (torch.einsum("hts,shd->thd", torch.softmax(s, -1), v.repeat_interleave(g, 1)).reshape(n, -1) @ self.attn_out.T)
        return self.norm(x, self.final) @ self.embed.T


# f32 arithmetic (sums of up to 256 terms: about 2^-18 of a hidden row) and f16 roundings that fall the other way for it (2^-11 of
# an element, one in 2^7): about 2^-15 of a row; logits of up to 16
TOL = 16 * 2.0 ** -15


@pytest.mark.parametrize("mix", [1.0, 0.02])  # drafts hardly ever right, and often
@pytest.mark.parametrize("lens,ways,drafts,steps", [((45, 9), 3, 3, 6), ((1,), 2, 5, 4), ((70, 8, 33), 1, 1, 9)])
def test_greedy_runs_are_the_models_own(ex, oracle_lib, lens, ways, drafts, steps, mix):
    c = type("C", (ex.Config,), dict(mix=mix))
    rng = np.random.default_rng(len(lens))
    prompts = [rng.integers(0, ex.Config.V, n).astype(np.int32) for n in lens]
    w = ex.Weights(seed=ways)
    res = ex.generate(w, prompts, ways, drafts, steps, temperature=0.0, c=c)
    assert ex.qg.device_status() == 0
    plain = Plain(w, c, oracle_lib, ex.gs)
    for prompt, lines in zip(prompts, res):
        assert len(lines) == ways
        for t in lines:
            assert steps < len(t) <= 1 + steps * (drafts + 1)
            x = plain.logits([*prompt.tolist(), *t[:-1]])[len(prompt) - 1:]
            best = x.max(-1).values
            assert (best - x[torch.arange(len(t)), torch.tensor(t)]).max() <= 2 * TOL


@pytest.mark.parametrize("mix", [1.0, 0.05, 1e-3])  # nearly all drafts refused, some, nearly none
def test_sampled_runs_follow_their_numbers(ex, oracle_lib, mix):
    rng = np.random.default_rng(7)
    c, temperature = type("C", (ex.Config,), dict(mix=mix)), 0.7
    prompts = [rng.integers(0, c.V, n).astype(np.int32) for n in (40, 3)]
    w = ex.Weights(seed=5)
    ways, drafts, steps = 4, 3, 5
    trace = []
    res = ex.generate(w, prompts, ways, drafts, steps, temperature=temperature, seed=3, c=c, trace=trace)
    assert ex.qg.device_status() == 0
    plain = Plain(w, c, oracle_lib, ex.gs)
    # a probability's relative error: two logits' over the temperature
    rel = 2 * TOL / temperature

    def drawn(r, u, token, slack):
        run = torch.cumsum(r, 0)
        want = u * run[-1]
        return run[token] >= want - slack and (run[token] - r[token]) <= want + slack

    total = 0
    for i in range(len(prompts) * ways):
        line, at = res[i // ways][i % ways], 0
        text = prompts[i // ways].tolist()
        p = torch.softmax(plain.logits([*text, *line])[len(text) - 1:] / temperature, -1)  # row k: what follows line[:k]
        assert drawn(p[0], trace[0]["u_next"][i].double(), line[0], rel)
        assert line[0] == int(trace[0]["next"][i])
        at = 1
        for t in trace[1:]:
            k = int(t["accepted"][i])
            total += k
            toks = t["tokens"][i].tolist()
            assert toks[0] == line[at - 1] and toks[1:1 + k] == line[at:at + k]
            for j in range(min(k + 1, drafts)):
                x = toks[j + 1]
                have, want = float(t["u"][i, j]) * float(t["q"][i, j, x]), float(p[at + j, x])
                assert have < want * (1 + rel) if j < k else have >= want * (1 - rel)
            r = p[at + k]
            if k < drafts:
                r = (r - t["q"][i, k].double()).clamp(min=0)
            token = int(t["next"][i])
            assert token == line[at + k]
            assert drawn(r, t["u_next"][i].double(), token, 2 * rel)
            at += k + 1
        assert at == len(line)
    most = len(prompts) * ways * steps * drafts
    assert total > most / 2 if mix < 0.01 else total < most / 2 if mix == 1.0 else True
