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
                S = torch.where(S.abs() < 2.0 ** -150, 0.0, S)  # states are f32: what is below its least value is gone
                held = S.norm(dim=1)
                u = beta[t][:, None] * (v[t] - torch.einsum("hij,hi->hj", S, k[t]))
                S = S + k[t][..., None] * u[:, None]
                out[t] = torch.einsum("hij,hi->hj", S, q[t])
                err = grow[t][:, None] * err + held + S.norm(dim=1) + v[t].abs() + 2.0 ** -149
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


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 128), (128, 256), (128, 64)])
@pytest.mark.parametrize("what", ["q", "k", "v", "a", "b"])
@pytest.mark.parametrize("at", [(2,), (45,), (100,), (145,), (40, 70), (31, 32, 149)], ids=str)
def test_nonfinite_tokens_of_long_prompts(qg, Dk, Dv, what, at):
    """A NaN or an infinity in the first, a middle and the last chunk of five, in chunks that follow one another and among
    chunks without: heads of 128 columns take such a chunk token by token between others on the tensor cores."""
    n = [150, 6, 70]
    for value in (float("nan"), float("inf"), -float("inf")):
        c = Followed(n, Dk=Dk, Dv=Dv, ins=[0, 1, 2], outs=[3, 4, 5], raw=False, seed=39)
        out, states, size, sizes = c.reference()
        h, j = 1, 33
        t = c.parts(c.x, c.ba)["qkvab".index(what)]
        cols = slice(j, j + 1) if what == "v" else slice(None)
        heads = [0, 1] if what in "qk" else [h]  # key head 0: value heads 0 and 1
        hit, shit = torch.zeros_like(out, dtype=torch.bool), torch.zeros_like(states, dtype=torch.bool)
        if what == "a" and value < 0:  # forgets everything: finite, and the reference knows it
            for i in at:
                t[i, h] = value
            c.check(c.run(qg))
            continue
        for i in at:
            if what in "qk":
                t[i, 0, 5] = value
            elif what == "v":
                t[i, h, j] = value
            else:
                t[i, h] = value
            for x in heads:
                hit[i:i + 1 if what == "q" else n[0], x, cols] = True
                if what != "q":
                    shit[3, x, :, cols] = True
        o, s = [x.double().cpu() for x in c.run(qg)]
        assert ((o - out).abs() <= 48 * 2.0 ** -24 * size * c.scale + 1e-37)[~hit].all()
        assert not torch.isfinite(o[hit]).any()
        assert ((s - states).abs() <= 48 * 2.0 ** -24 * sizes + 1e-37)[~shit].all()
    assert qg.device_status() == 0


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 256)])
def test_extremes_of_whole_columns(qg, Dk, Dv):
    """Heads of whole 128 columns: no decay and decays that leave nothing, steps of 0 to 2, zero rows, columns of 10^25 and 10^-30
    beside others, states that are not finite."""
    c = Delta([90], Dk=Dk, Dv=Dv, raw=False, ins=[0], outs=[1], seed=40)
    g = torch.Generator().manual_seed(41)
    kinds = torch.tensor([0.0, -float("inf"), -1e30, -104.0, -12.0, -1e-6])
    c.ba[:, :c.Hv] = kinds[torch.randint(0, len(kinds), (90, c.Hv), generator=g)]
    c.ba[:, 0], c.ba[:, 1] = 0.0, -11.0
    c.ba[:, c.Hv:2 * c.Hv] = torch.tensor([0.0, 1.0, 0.5, 2.0])[torch.randint(0, 4, (90, c.Hv), generator=g)]
    c.check(c.run(qg))
    for big in (1e-30, 1e25):
        c = Delta([50, 2], Dk=Dk, Dv=Dv, ins=[0, 1], outs=[2, 3], seed=42)
        f = torch.where(torch.arange(Dv) % 2 == 0, big, 1.0)
        c.states *= f
        c.parts(c.x, c.ba)[2].mul_(f)
        c.check(c.run(qg))
    c = Delta([40, 1], Dk=Dk, Dv=Dv, ins=[0, 1], outs=[2, 3], seed=43)
    q, k, v, _, _ = c.parts(c.x, c.ba)
    q[3], k[7], k[40], v[9] = 0, 0, 0, 0
    c.check(c.run(qg))
    c = Delta([100, 40], Dk=Dk, Dv=Dv, ins=[0, 1], outs=[2, 3], seed=44)
    out, _, size, _ = c.reference()
    c.states[0, 1, 3, 7], c.states[1, 0, 9, 40] = float("inf"), float("nan")
    o = c.run(qg)[0].double().cpu()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:100, 1, 7] = hit[100:, 0, 40] = True
    assert ((o - out).abs() <= 48 * 2.0 ** -24 * size * c.scale + 1e-37)[~hit].all() and not torch.isfinite(o[hit]).any()
    assert qg.device_status() == 0


@pytest.mark.parametrize("Dv", [128, 64])
def test_starts_that_do_not_rise_write_nothing_else(qg, Dv):
    """Starts that are negative, fall or pass the rows: rows around, slots that nobody is given and what lies behind the workspace stay
    as they were."""
    c = Delta([20, 20, 20], Dv=Dv, ins=[0, 1, 2], outs=[3, 4, 5], seed=45)
    hold = []
    c.run(qg, hold=hold)
    args, kw = list(hold[0]), dict(hold[1])
    kw["q_start"] = torch.tensor([-5, 70, 30, 1000], dtype=torch.int32, device="cuda")
    kw["max_new"] = 0
    out = torch.full((c.T + 64, c.Hv, c.Dv), 7.5, device="cuda")
    pool = torch.randn((c.slots + 4, c.Hv, c.Dk, c.Dv), device="cuda")
    pool[2:2 + c.slots] = c.states.cuda()
    need = qg.delta_workspace_size(c.T, 3, c.Hk, c.Hv, c.Dk, c.Dv)
    ws = torch.full((need + 4096,), 90, dtype=torch.uint8, device="cuda")
    before = pool.clone()
    args[5], args[8], args[9] = pool[2:2 + c.slots], out[32:32 + c.T], ws[:need]
    qg.delta_rule(*args, **kw)
    torch.cuda.synchronize()
    assert (out[:32] == 7.5).all() and (out[32 + c.T:] == 7.5).all() and (ws[need:] == 90).all()
    kept = [i for i in range(c.slots + 4) if i - 2 not in (3, 5)]  # the second sequence has no rows
    assert torch.equal(pool[kept], before[kept])
    assert qg.device_status() == 0


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 256), (128, 64), (64, 32)])
@pytest.mark.parametrize("reset", [-float("inf"), -200.0, -110.0])
def test_what_is_forgotten_does_not_grow_back(qg, Dk, Dv, reset):
    """A decay that leaves nothing, then log decays that add up to more than it took in the same chunk and the next: without
    new values the state stays 0, and with them it is theirs."""
    for n, at in (([60], 3), ([60], 40), ([12], 3)):
        for later, first in ((0.0, 60.0), (0.0, 30.0), (1.0, 5.0)):
            c = Followed(n, Dk=Dk, Dv=Dv, raw=False, ins=[0], outs=[1], seed=46)
            c.ba[:, :c.Hv] = -0.1
            c.ba[at, :c.Hv] = reset
            c.ba[at + 1:, :c.Hv] = 0.5
            c.ba[at + 1:at + 3, :c.Hv] = first
            c.parts(c.x, c.ba)[2][at:] *= later
            c.check(c.run(qg))
    assert qg.device_status() == 0
