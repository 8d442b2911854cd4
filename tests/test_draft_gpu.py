"""Probabilities and draft verification on the GPU against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


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


# ---- probabilities ------------------------------------------------------------------------------

def probs_reference(x, temp):
    """p in 64 bits, and the exponent that each came from."""
    x = x.double().clone()
    x[torch.isnan(x)] = -math.inf
    out, power = torch.zeros_like(x), torch.zeros_like(x)
    for r in range(x.shape[0]):
        m = x[r].max()
        t = 1.0 if temp is None else float(temp[r])
        if math.isinf(m):
            continue
        if not t > 0:
            out[r, int((x[r] == m).nonzero()[0])] = 1
            continue
        d = (x[r] - m) / t if not math.isinf(t) else torch.where(x[r] == -math.inf, -math.inf, 0.0)
        power[r] = d
        e = torch.exp(d)
        out[r] = e / e.sum()
    return out, power


def check_probs(got, x, temp):
    """A probability's exponent is off by 3 roundings of its size, twice (against a slice's maximum and between slices); the two
    exponentials, their product and the quotient by 8 more, the sum of positive terms by one for each it passes through: n / 512
    in a thread's turn, 5 in a warp, 16 warps, 8 slices."""
    want, power = probs_reference(x.cpu(), temp)
    V = x.shape[1]
    tol = want * U * (6 * power.clamp(min=-200).abs() + 8 + V / 512 + 29) + 2.0 ** -126
    err = (got.double().cpu() - want).abs()
    assert err.le(tol).all(), (err / tol).max()


@pytest.mark.parametrize("V", [1, 2, 3, 5, 127, 1000, 4097, 16389, 151936, 262147])
@pytest.mark.parametrize("T", [1, 3])
def test_probs_sizes(qg, V, T):
    g = torch.Generator().manual_seed(V)
    x = 3 * torch.randn((T, V), generator=g)
    for temp in (None, torch.tensor([0.7, 1.9, 0.0])[:T]):
        out = torch.full((T, V), float("nan"), device="cuda")
        qg.token_probs(x.cuda(), out, temperature=None if temp is None else temp.cuda())
        check_probs(out, x, temp)


def test_probs_largest_vocabulary(qg):
    """More than the shared memory of a row's blocks holds, in place as well."""
    V = 1 << 20
    x = 2 * torch.randn((2, V), generator=torch.Generator().manual_seed(0))
    d = x.cuda()
    out = torch.empty_like(d)
    qg.token_probs(d, out)
    check_probs(out, x, None)
    qg.token_probs(d, d)
    assert torch.equal(d, out)


@pytest.mark.parametrize("T,V", [(90, 90004), (83, 163836), (300, 81940)])
def test_probs_many_rows(qg, T, V):
    """Rows that clusters take in turn, in place as well, with greedy rows, rows without a distribution and odd values among them."""
    g = torch.Generator().manual_seed(T)
    x = 3 * torch.randn((T, V), generator=g)
    temp = 0.3 + torch.rand((T,), generator=g)
    temp[::7] = 0.0
    x[3], x[11, 5], x[20, ::3] = -math.inf, math.nan, torch.finfo(torch.float32).min
    x[14, V - 1] = x[14, 9] = 50.0  # a greedy row with a tie
    x[30, 7] = math.inf
    out = torch.full((T, V), math.nan, device="cuda")
    d = x.cuda()
    qg.token_probs(d, out, temperature=temp.cuda())
    check_probs(out, x, temp)
    qg.token_probs(d, d, temperature=temp.cuda())
    assert torch.equal(d, out)
    assert qg.device_status() == 0


@pytest.mark.parametrize("V", [7, 5003, 60000])
def test_probs_special_rows(qg, V):
    lo, inf, nan = torch.finfo(torch.float32).min, math.inf, math.nan
    rows = [torch.randn(V, generator=torch.Generator().manual_seed(i)) for i in range(12)]
    rows[0][:] = -inf                      # nothing allowed: zeros
    rows[1][:] = lo                        # the lowest value everywhere: equal shares
    rows[2][1:] = -inf                     # one token
    rows[3][::2] = lo
    rows[4][2] = inf                       # no distribution: zeros
    rows[5][3] = nan                       # counts as -inf
    rows[6][:] = nan
    rows[7][V // 2] = torch.finfo(torch.float32).max
    rows[7][0] = lo
    rows[8][:-1] = -inf                    # the last one
    rows[9][1:3] = 9.0                     # a tie for the greedy pick: the lowest
    rows[10][:] = 5.0
    x = torch.stack(rows)
    for t in (1.0, 0.0, -1.0, nan, 1e-39, 3e38, inf, 0.01):
        temp = torch.full((12,), t)
        out = torch.full((12, V), nan, device="cuda")
        qg.token_probs(x.cuda(), out, temperature=temp.cuda())
        assert torch.isfinite(out).all()
        if t == 1e-39:  # a quotient by it leaves f32: what is below the largest is 0
            want = (x == torch.nan_to_num(x, nan=-inf, posinf=inf, neginf=-inf).amax(1, keepdim=True)).double()
            want[torch.isinf(torch.nan_to_num(x, nan=-inf, posinf=inf, neginf=-inf).amax(1))] = 0
            want = torch.nan_to_num(want / want.sum(1, keepdim=True))
            assert (out.double().cpu() - want).abs().max() <= 1e-5
        else:
            check_probs(out, x, temp)


# ---- verification -----------------------------------------------------------------------------------

def clean(p):
    p = np.asarray(p, dtype=np.float32)
    return np.minimum(np.where(p > 0, p, np.float32(0)), np.float32(2.0 ** 100))


def verify_reference(p, q, tokens, u, u_next, start, kv=None):
    acc, tok, kept, V = [], [], [], p.shape[1]
    for b in range(len(start) - 1):
        s, e = start[b], start[b + 1]
        if e <= s:
            acc.append(0), tok.append(-1), kept.append(None if kv is None else kv[b])
            continue
        t = s
        while t + 1 < e:
            x = int(tokens[t + 1])
            if not 0 <= x < V:
                break
            pp, qq = float(clean(p[t, x])), 1.0 if q is None else float(clean(q[t, x]))
            uu = float(u[t]) if u[t] > 0 else 0.0
            if not uu * qq < pp:
                break
            t += 1
        row = clean(p[t])
        r = row.copy()
        if t + 1 < e:
            if q is not None:
                r = np.maximum(row - clean(q[t]), np.float32(0))
            elif 0 <= tokens[t + 1] < V:
                r[tokens[t + 1]] = max(np.float32(0), r[tokens[t + 1]] - np.float32(1))
        if not r.sum(dtype=np.float64) > 0:
            r = row
        c = np.cumsum(r.astype(np.longdouble))
        want = (np.longdouble(u_next[b]) if u_next[b] > 0 else np.longdouble(0)) * c[-1]
        over = np.nonzero((c > want) & (r > 0))[0]
        some = np.nonzero(r > 0)[0]
        acc.append(t - s)
        tok.append(int(over[0]) if len(over) else int(some[-1]) if len(some) else -1)
        kept.append(None if kv is None else kv[b] - (e - 1 - t))
    return acc, tok, kept


def run_verify(qg, p, q, tokens, u, u_next, start, kv=None, plain_start=False):
    up = lambda a, t: None if a is None else torch.as_tensor(np.asarray(a), dtype=t, device="cuda").contiguous()  # noqa: E731
    f32, i32, B = torch.float32, torch.int32, len(start) - 1
    acc, tok = (torch.full((B,), -7, dtype=i32, device="cuda") for _ in range(2))
    kept = None if kv is None else torch.full((B,), -7, dtype=i32, device="cuda")
    qg.draft_verify(up(p, f32), up(tokens, i32), up(u, f32), up(u_next, f32), acc, tok, draft_probs=up(q, f32),
                    q_start=None if plain_start else up(start, i32), kv_len=up(kv, i32), kept_len=kept)
    return acc.tolist(), tok.tolist(), [None] * B if kv is None else kept.tolist()


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def drafted(rng, n, V, sharp=2.0, near=0.6):
    rows = [x + 1 for x in n]
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    T = int(start[-1])
    x = sharp * rng.standard_normal((T, V))
    p, q = softmax(x + near * rng.standard_normal((T, V))), softmax(x)
    tokens = np.zeros(T, np.int32)
    for t in range(T - 1):
        tokens[t + 1] = min(V - 1, int(np.searchsorted(np.cumsum(q[t].astype(np.float64)), rng.random() * 0.999999)))
    return p, q, tokens, rng.random(T).astype(np.float32), rng.random(len(n)).astype(np.float32), start


@pytest.mark.parametrize("V", [1, 2, 3, 4, 7, 63, 1001, 4098, 9001, 40003])
@pytest.mark.parametrize("certain", [False, True])
def test_verify_sizes(qg, V, certain):
    rng = np.random.default_rng(V)
    for n in ([0], [3], [4, 0, 1, 7, 2], [1] * 9):
        p, q, tokens, u, un, start = drafted(rng, n, V)
        q = None if certain else q
        kv = [50 + x for x in n]
        assert run_verify(qg, p, q, tokens, u, un, start, kv) == verify_reference(p, q, tokens, u, un, start, kv)
    assert qg.device_status() == 0


@pytest.mark.parametrize("B", [1, 5, 150, 400])
def test_verify_draws_every_place(qg, B):
    """Random numbers all over [0, 1): blocks', warps' and threads' borders among them."""
    V = 20011
    rng = np.random.default_rng(B)
    p = softmax(0.1 * rng.standard_normal((B, V)))
    un = ((np.arange(B) + 0.5) / B).astype(np.float32)
    start = np.arange(B + 1)
    want = verify_reference(p, None, np.zeros(B, np.int32), np.zeros(B), un, start)
    assert run_verify(qg, p, None, np.zeros(B), np.zeros(B), un, start) == want
    assert run_verify(qg, p, None, np.zeros(B), np.zeros(B), un, start, plain_start=True) == want
    # a sampler without tokens and random numbers for drafts
    acc, tok = (torch.empty((B,), dtype=torch.int32, device="cuda") for _ in range(2))
    qg.draft_verify(torch.from_numpy(p).cuda(), None, None, torch.from_numpy(un).cuda(), acc, tok)
    assert tok.tolist() == want[1] and acc.tolist() == [0] * B


def test_verify_borders(qg):
    """Thresholds that fall exactly on sums: the sum has to be larger, so the next token with mass is drawn."""
    V = 8192
    p = np.zeros((6, V), np.float32)
    p[:, [3, 700, 4096, 8191]] = 0.25
    un = np.array([0.0, 0.25, 0.5, 0.75, 1.0, 7.0], np.float32)
    got = run_verify(qg, p, None, np.zeros(6), np.zeros(6), un, np.arange(7))
    assert got[1] == [3, 700, 4096, 8191, 8191, 8191]
    # equality does not accept; u = 0 accepts whatever has mass, never what has none
    p = np.full((6, 8), 0.125, np.float32)
    q = np.full((6, 8), 0.25, np.float32)
    p[2, 5] = 0.0
    tokens = np.array([0, 5, 0, 5, 0, 5], np.int32)
    u = np.array([0.5, 0, 0.0, 0, 0.4999, 0], np.float32)
    start = np.array([0, 2, 4, 6])
    assert run_verify(qg, p, q, tokens, u, [0.0] * 3, start)[0] == [0, 0, 1]


def test_verify_nothing_left(qg):
    """The drafter's probabilities above the target's everywhere: drawn from the target's; rows without mass: -1."""
    V = 5000
    rng = np.random.default_rng(3)
    p = softmax(rng.standard_normal((4, V)))
    q = np.minimum(p * 2, 1).astype(np.float32)
    p[2:] = 0
    tokens = np.array([0, 11, 0, 11], np.int32)
    u = np.full(4, 0.9999, np.float32)
    start = np.array([0, 2, 4])
    got = run_verify(qg, p, q, tokens, u, [0.37, 0.5], start)
    assert got == verify_reference(p, q, tokens, u, [0.37, 0.5], start)
    assert got[1][1] == -1 and got[0] == [0, 0]


@pytest.mark.parametrize("V", [9, 6001])
def test_verify_odd_values(qg, V):
    """NaN, negative and infinite probabilities and random numbers, tokens outside the vocabulary, empty sequences."""
    rng = np.random.default_rng(V)
    n = [3, 2, 2, 4, 2]
    p, q, tokens, u, un, start = drafted(rng, n, V, near=0.2)
    p[0, ::3], p[1, 1], q[0, ::2], p[4, 2] = np.nan, -1.0, -np.inf, np.inf
    q[8, :], u[0], u[5], un[1], un[2] = np.nan, -3.0, np.nan, np.nan, -1.0
    assert run_verify(qg, p, q, tokens, u, un, start) == verify_reference(p, q, tokens, u, un, start)
    assert qg.device_status() == 0
    tokens[start[0] + 1], tokens[start[3] + 2], u[:] = V, -1, 0.0
    start = np.insert(start, 2, start[2])  # a sequence without rows
    un = np.insert(un, 1, 0.5)
    kv = list(range(60, 66))
    got = run_verify(qg, p, q, tokens, u, un, start, kv)
    assert got == verify_reference(p, q, tokens, u, un, start, kv)
    assert qg.device_status() == 1 << qg.QG_EDEVICE_ID


def test_verify_far_rows(qg):
    """Rows whose offsets pass 32 bits."""
    V = 1 << 20
    T = 2 ** 31 // V + 3
    p = torch.zeros((T, V), device="cuda")
    p[:, 77] = 1.0
    p[T - 1] = 0.0
    p[T - 1, V - 2] = 0.5
    acc, tok = (torch.empty((2,), dtype=torch.int32, device="cuda") for _ in range(2))
    tokens = torch.full((T,), 77, dtype=torch.int32, device="cuda")
    u = torch.full((T,), 0.5, device="cuda")
    q_start = torch.tensor([0, 1, T], dtype=torch.int32, device="cuda")
    qg.draft_verify(p, tokens, u, torch.tensor([0.1, 0.9], device="cuda"), acc, tok, q_start=q_start)
    assert acc.tolist() == [0, T - 2] and tok.tolist() == [77, V - 2]


def test_bad_starts_stay_inside(qg):
    p = torch.full((6, 50), 0.02, device="cuda")
    acc, tok = (torch.empty((3,), dtype=torch.int32, device="cuda") for _ in range(2))
    q_start = torch.tensor([-4, 90, 2, 7], dtype=torch.int32, device="cuda")
    qg.draft_verify(p, torch.zeros(6, dtype=torch.int32, device="cuda"), torch.zeros(6, device="cuda"), torch.zeros(3, device="cuda"),
                    acc, tok, q_start=q_start)
    torch.cuda.synchronize()
    assert all(-1 <= x < 50 for x in tok.tolist())


def test_graph_and_stream(qg):
    """Both calls captured in one graph and replayed on new logits; another stream gives the same."""
    rng = np.random.default_rng(5)
    n, V = [3, 1, 2], 12345
    p, q, tokens, u, un, start = drafted(rng, n, V)
    T = p.shape[0]
    d = lambda a, t=torch.float32: torch.as_tensor(a, dtype=t, device="cuda")  # noqa: E731
    logits, probs = torch.log(d(p)).clamp(min=-80), torch.empty((T, V), device="cuda")
    q, tokens_d, u, un = d(q), d(tokens, torch.int32), d(u), d(un)
    start_d = d(start, torch.int32)
    acc, tok = (torch.empty((3,), dtype=torch.int32, device="cuda") for _ in range(2))

    def step(stream=None):
        qg.token_probs(logits, probs, stream=stream)
        qg.draft_verify(probs, tokens_d, u, un, acc, tok, draft_probs=q, q_start=start_d, stream=stream)

    step()
    want = acc.tolist(), tok.tolist()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.synchronize()
    assert (acc.tolist(), tok.tolist()) == want
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    logits.copy_(torch.randn((T, V), device="cuda"))
    un.copy_(torch.rand(3, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    ref = verify_reference(probs.cpu().numpy(), q.cpu().numpy(), tokens, u.cpu().numpy(), un.cpu().numpy(), start)
    assert (acc.tolist(), tok.tolist()) == ref[:2]


@pytest.mark.parametrize("V", [9, 6001])
@pytest.mark.parametrize("token", [-1, None])
def test_a_drafted_token_outside_the_vocabulary(qg, V, token):
    """It is not accepted: with a drafter's probabilities the difference is drawn from, with certain drafts the target's whole row."""
    rng = np.random.default_rng(V)
    p, q, tokens, _, _, start = drafted(rng, [2, 2], V)
    tokens[1] = tokens[5] = V if token is None else token
    u, un = np.zeros(6, np.float32), np.array([0.999, 0.001], np.float32)
    got = run_verify(qg, p, q, tokens, u, un, start)
    assert got == verify_reference(p, q, tokens, u, un, start) and got[0] == [0, 1]
    rest = np.maximum(p[0] - q[0], 0)
    assert rest[got[1][0]] > 0
    assert qg.device_status() == 1 << qg.QG_EDEVICE_ID
    got = run_verify(qg, p, None, tokens, u, un, start)
    assert got == verify_reference(p, None, tokens, u, un, start) and got[0] == [0, 1]
    assert run_verify(qg, p[[0, 4]], None, np.zeros(2), np.zeros(2), un, [0, 1, 2])[1] == got[1]  # the rows as a sampler takes them
    assert qg.device_status() == 1 << qg.QG_EDEVICE_ID
