"""The gated delta rule over prompts: where the chunks could go wrong, against the definition in 64 bits."""
import pytest
import torch

from drafted_helpers import Delta

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gguf_block_dequant_gb300 as qg
    from gguf_block_dequant_gb300 import build

    build.build()
    qg.load()
    qg.device_status()
    return qg


class Followed(Delta):
    """A call whose bound follows the state: what a token adds (the helpers' 48 roundings of its column's length) is carried on
    by e^g max(1, |1 - beta |k|^2|), the most that a later token makes of it, so that it shrinks when the state is
    forgotten and grows when the state does.  It never looks at later tokens."""

    def reference(self):
        q, k, v, a, b = [t.double() for t in self.parts(self.x, self.ba)]
        if self.l2:
            q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + 1e-6)
            k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + 1e-6)
        g, beta = a, b
        if self.raw:
            g = self.a_scale.double() * torch.logaddexp(a + self.a_bias.double(), torch.zeros_like(a))
            beta = torch.sigmoid(b)
        key = [h % self.Hk if self.tiled else h // (self.Hv // self.Hk) for h in range(self.Hv)]
        q, k = q[:, key] * self.scale, k[:, key]
        grow = torch.exp(g) * (1 - beta * k.square().sum(-1)).abs().clamp(min=1)
        out = torch.full((self.T, self.Hv, self.Dv), float("nan"), dtype=torch.float64)
        states, size, sizes = self.states.double(), torch.zeros_like(out), torch.zeros(self.slots, self.Hv, 1, self.Dv).double()
        before = states.clone()
        for s, n in enumerate(self.n):
            at = self.ins[s] if self.ins else -1
            S = before[at].clone() if at >= 0 else torch.zeros_like(states[0])
            err = torch.zeros_like(size[0])
            for t in range(self.start[s], self.start[s] + n):
                S = torch.exp(g[t])[:, None, None] * S
                held = S.norm(dim=1)
                u = beta[t][:, None] * (v[t] - torch.einsum("hij,hi->hj", S, k[t]))
                S = S + k[t][..., None] * u[:, None]
                out[t] = torch.einsum("hij,hi->hj", S, q[t])
                err = grow[t][:, None] * err + held + S.norm(dim=1) + v[t].abs()
                size[t] = err
            if n and self.outs and self.outs[s] >= 0:
                states[self.outs[s]], sizes[self.outs[s], :, 0] = S, err
        return out, states, size, sizes


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 128), (128, 64), (64, 32)])
@pytest.mark.parametrize("g", [0.005, 0.05, 0.3])
def test_states_that_grow(qg, Dk, Dv, g):
    """Positive log decays: the factors of a chunk are above 1, up to e^12, and those of one head go both ways."""
    for n in ([6], [90, 40], [20]):
        B = len(n)
        c = Followed(n, Dk=Dk, Dv=Dv, raw=False, ins=list(range(B)), outs=list(range(B, 2 * B)), seed=31)
        r = torch.rand((c.T, c.Hv), generator=torch.Generator().manual_seed(32))
        c.ba[:, :c.Hv] = g * (0.5 + r)
        c.ba[:, 1] = 8 * g * (r[:, 1] - 0.5)
        c.check(c.run(qg))
    c = Followed([70], Dk=Dk, Dv=Dv, ins=[0], outs=[1], seed=33)  # raw gates under a positive factor
    c.a_scale = torch.full((c.Hv,), g)
    c.check(c.run(qg))
    assert qg.device_status() == 0


@pytest.mark.parametrize("hint", [0, 1, 64])
def test_the_hint_changes_nothing_where_states_grow(qg, hint):
    """max_new below, at and above what the sequence has: token by token and in chunks alike."""
    c = Followed([64], raw=False, ins=[0], outs=[1], seed=34)
    c.ba[:, :c.Hv] = 0.1
    c.check(c.run(qg, max_new=hint))


def by_place(c, f):
    """Values times f of a token's place in its chunk of 32."""
    v = c.parts(c.x, c.ba)[2]
    for s, n in enumerate(c.n):
        for t in range(n):
            v[c.start[s] + t] *= f[t % 32]


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 128), (128, 64), (64, 32)])
@pytest.mark.parametrize("power", [6, 12, 30])
def test_magnitudes_within_a_chunk(qg, Dk, Dv, power):
    """Values that grow by up to 10^30 within a chunk, from states of zeros: earlier tokens keep their own precision.  Values that
    shrink as much, under decays that forget them: later tokens have theirs."""
    f = torch.logspace(-power / 2, power / 2, 32, dtype=torch.float64).float()
    for n in ([32], [20, 96, 70]):
        B = len(n)
        c = Followed(n, Dk=Dk, Dv=Dv, ins=[-1] * B, outs=list(range(B)), seed=35)
        by_place(c, f)
        c.check(c.run(qg))
        c = Followed(n, Dk=Dk, Dv=Dv, raw=False, ins=[-1] * B, outs=list(range(B)), seed=36)
        by_place(c, f.flip(0))
        c.ba[:, :c.Hv] = -11.0
        c.ba[:, 0] = -2.5
        c.check(c.run(qg))
    assert qg.device_status() == 0


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("reset", [-float("inf"), -40.0])
def test_a_state_forgotten_within_a_chunk(qg, Dk, Dv, reset):
    """A state of 10^6 and the values before a token that forgets them do not cost the tokens behind it their precision."""
    for at in (0, 3, 31, 40, 63):
        c = Followed([70], Dk=Dk, Dv=Dv, raw=False, ins=[0], outs=[1], seed=37)
        c.states[0] *= 1e6
        c.parts(c.x, c.ba)[2][:at] *= 1e6
        c.ba[:, :c.Hv] = -0.01
        c.ba[at, :c.Hv] = reset
        c.check(c.run(qg))


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 256), (128, 64), (64, 32)])
@pytest.mark.parametrize("what", ["v", "k", "growth", "largest"])
def test_an_overflow_reaches_no_earlier_token(qg, Dk, Dv, what):
    """Finite inputs whose updates or states leave f32: tokens before the first that does keep their results, and other columns all."""
    for n, at in (([70, 40], 5), ([70, 40], 40), ([64], 60)):
        B = len(n)
        c = Followed(n, Dk=Dk, Dv=Dv, raw=False, l2=False, ins=list(range(B)), outs=list(range(B, 2 * B)), seed=38)
        q, k, v, a, b = c.parts(c.x, c.ba)
        h, j, cols = 1, 17, slice(None)
        if what == "v":  # the step doubles it
            v[at, h, j], b[at, h], cols = 3e38, 2.0, slice(17, 18)
        elif what == "largest":  # next to f32's largest, and taken twice by the keys of the next token
            v[at, h, j], b[at, h], cols = torch.finfo(torch.float32).max, 1.0, slice(17, 18)
        elif what == "k":  # key head 0: value heads 0 and 1
            k[at:at + 2, 0] *= 1e25
        else:
            a[at:at + 3, h] = 60.0
        out, states, size, _ = c.reference()
        o, s = [t.double().cpu() for t in c.run(qg)]
        ok = (o - out).abs() <= 48 * 2.0 ** -24 * size * c.scale + 1e-37
        hit = torch.zeros_like(ok)
        hit[at:n[0], 0 if what == "k" else h:h + 1, cols] = True
        hit[at:n[0], h, cols] = True
        assert ok[~hit].all()
        assert torch.isfinite(o[~hit]).all()
        if what != "largest":
            assert not torch.isfinite(o[min(at + 3, n[0] - 1), h, j])
        for x in range(c.Hv):
            if x != h and not (what == "k" and x == 0):
                assert (s[B, x] - states[B, x]).abs().max() <= 1e-3
    assert qg.device_status() == 0
