"""64-bit references of the drafted-decode tests, on the CPU."""
import math

import torch

EPS = 1e-6
U = 2.0 ** -24  # half a step of f32, relative


class Delta:
    """A call of the gated delta rule on the GPU, and what it has to give.  `n`: tokens per sequence; `ins`, `outs`: slots (None: no
    array); q, k, v and both gates are slices of wider rows, `behind` rows follow the last sequence."""

    def __init__(self, n, Hk=2, Hv=4, Dk=128, Dv=128, raw=True, l2=True, tiled=False, ins=None, outs=None, each=None, slots=None,
                 behind=0, seed=0, wide=8):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.n, self.Hk, self.Hv, self.Dk, self.Dv, self.raw, self.l2, self.tiled = list(n), Hk, Hv, Dk, Dv, raw, l2, tiled
        self.start = [0]
        for x in n:
            self.start.append(self.start[-1] + x)
        T = self.start[-1] + behind
        self.T, self.ins, self.outs, self.each = T, ins, outs, each
        x = r(T, 2 * Hk * Dk + Hv * Dv + wide)
        if not l2:
            x[:, :2 * Hk * Dk] /= x[:, :2 * Hk * Dk].view(T, 2 * Hk, Dk).norm(dim=-1).repeat_interleave(Dk, 1)
        self.x, self.ba = x, r(T, 2 * Hv + 3)
        self.a_scale = -torch.exp(math.log(16.0) * torch.rand(Hv, generator=g)) if raw else None
        self.a_bias = 2.0 * r(Hv) - 4.0 if raw else None
        if not raw:
            self.ba[:, :Hv] = -torch.exp(self.ba[:, :Hv] - 2.0)
            self.ba[:, Hv:2 * Hv] = torch.rand((T, Hv), generator=g)
        used = [s for lst in (ins, outs, each) if lst is not None for s in lst]
        self.slots = slots or max([0, *used]) + 2
        self.states = r(self.slots, Hv, Dk, Dv)
        self.scale = Dk ** -0.5

    def parts(self, x, ba):
        Hk, Hv, Dk, Dv = self.Hk, self.Hv, self.Dk, self.Dv
        a, b = Hk * Dk, 2 * Hk * Dk
        return (x[:, :a].unflatten(1, (Hk, Dk)), x[:, a:b].unflatten(1, (Hk, Dk)), x[:, b:b + Hv * Dv].unflatten(1, (Hv, Dv)),
                ba[:, :Hv], ba[:, Hv:2 * Hv])

    def run(self, qg, max_new=None, fill=float("nan"), stream=None, states=None, hold=None):
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        x, ba = self.x.cuda(), self.ba.cuda()
        states = self.states.cuda() if states is None else states
        out = torch.full((self.T, self.Hv, self.Dv), fill, device="cuda")
        one = all(c == 1 for c in self.n) and self.T == len(self.n)
        q_start = None if one else i32(self.start)
        most = max(self.n) if max_new is None else max_new
        ws = torch.full((max(16, qg.delta_workspace_size(self.T, len(self.n), self.Hk, self.Hv, self.Dk, self.Dv, most)),), 255,
                        dtype=torch.uint8, device="cuda")
        args = (*self.parts(x, ba), states, i32(self.ins), i32(self.outs), out, ws)
        kw = dict(q_start=q_start, max_new=most, state_each=i32(self.each), a_scale=dev(self.a_scale), a_bias=dev(self.a_bias),
                  l2norm_eps=EPS if self.l2 else None, scale=self.scale, tiled=self.tiled)
        if hold is not None:
            hold += [args, kw]
        qg.delta_rule(*args, **kw, stream=stream)
        return out, states

    def reference(self):
        """(out, states) in 64 bits, and per element of each how large what is summed there gets."""
        q, k, v, a, b = [t.double() for t in self.parts(self.x, self.ba)]
        if self.l2:
            q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + EPS)
            k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + EPS)
        g, beta = a, b
        if self.raw:
            g = self.a_scale.double() * torch.logaddexp(a + self.a_bias.double(), torch.zeros_like(a))
            beta = torch.sigmoid(b)
        key = [h % self.Hk if self.tiled else h // (self.Hv // self.Hk) for h in range(self.Hv)]
        q, k = q[:, key] * self.scale, k[:, key]
        out = torch.full((self.T, self.Hv, self.Dv), float("nan"), dtype=torch.float64)
        states, size, sizes = self.states.double(), torch.zeros_like(out), torch.zeros(self.slots, self.Hv, 1, self.Dv).double()
        before = states.clone()
        for s, n in enumerate(self.n):
            at = self.ins[s] if self.ins else -1
            S = before[at].clone() if at >= 0 else torch.zeros_like(states[0])
            big = S.norm(dim=1)  # [Hv][Dv]: a column's length, the largest so far
            for t in range(self.start[s], self.start[s] + n):
                S = torch.exp(g[t])[:, None, None] * S
                u = beta[t][:, None] * (v[t] - torch.einsum("hij,hi->hj", S, k[t]))
                S = S + k[t][..., None] * u[:, None]
                out[t] = torch.einsum("hij,hi->hj", S, q[t])
                big = torch.maximum(big, S.norm(dim=1) + v[t].abs())
                size[t] = big * (t - self.start[s] + 1)
                if self.each and self.each[t] >= 0:
                    states[self.each[t]], sizes[self.each[t], :, 0] = S, size[t]
            if n and self.outs and self.outs[s] >= 0:
                states[self.outs[s]], sizes[self.outs[s], :, 0] = S, size[self.start[s] + n - 1]
        return out, states, size, sizes

    def check(self, got):
        """A token adds at most 48 roundings of a column's length (sums of 16 rows, 5 exchanges and 8 warps, norms, gates and the
        products; in chunks: operands within 2^-22, sums of 12 products within 2^-23 each, over 32 tokens), and what
        earlier ones left does not grow: e^g (1 - beta k k^T) is no larger than 1 for |k| <= 1.  The state's entries
        are bounded by its column, the outputs by the column times |scale q|."""
        out, states, size, sizes = self.reference()
        live = self.start[-1]
        o, s = [t.double().cpu() for t in got]
        # |q| is 1: an output sees the scale, and one rounding more
        assert (o[:live] - out[:live]).abs().le(48 * U * size[:live] * self.scale + 1e-37).all(), \
            ((o[:live] - out[:live]).abs() / (size[:live] * self.scale * U + 1e-37)).max()
        assert torch.isnan(o[live:]).all()  # rows behind the last sequence
        assert (s - states).abs().le(48 * U * sizes + 1e-37).all(), ((s - states).abs() / (sizes * U + 1e-37)).max()
        same = sizes[:, 0, 0, 0] == 0
        assert torch.equal(s[same], self.states.double()[same])  # slots that nobody writes
