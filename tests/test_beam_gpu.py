"""Beam selection against its definition in 64 bits: order, ties, ended beams, banned tokens,
rows without a distribution, sizes around the slices."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gguf_block_dequant_gb300 as qg
    from gguf_block_dequant_gb300 import build

    build.build()
    qg.load()
    return qg


def select(qg, logits, scores, N, W, K, done=None, eos=-1):
    V = logits.shape[-1]
    s = torch.full((N, K), float("nan"), device="cuda")
    p, t = (torch.full((N, K), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    d = torch.full((N, K), 9, dtype=torch.uint8, device="cuda")
    n = qg.beam_workspace_size(N, W, K, V)
    ws = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    qg.beam_select(logits, scores, N, W, s, p, t, ws[:n], done=done, eos=eos, done_out=d)
    torch.cuda.synchronize()
    assert (ws[n:] == 0xA5).all()
    return s.cpu(), p.cpu(), t.cpu(), d.cpu()


def ref_select(logits, scores, N, W, K, done=None, eos=-1):
    V = logits.shape[-1]
    x = logits.double().cpu()
    x = torch.where(torch.isnan(x), -math.inf, x)
    sc = scores.double().cpu()
    # the maximum is taken off first: a row at the type's lowest value would absorb the log of its sum
    m = x.amax(-1, keepdim=True)
    lp = (x - m) - torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    lp = torch.where(torch.isnan(lp), -math.inf, lp)
    if done is not None:
        only = torch.full((V,), -math.inf, dtype=torch.float64)
        if eos >= 0:
            only[eos] = 0
        lp = torch.where(done.cpu().bool()[:, None], only, lp)
    sc = torch.where(torch.isfinite(sc), sc, -math.inf)
    cand = (sc[:, None] + lp).view(N, W * V)
    val, idx = torch.sort(cand, dim=-1, descending=True, stable=True)
    val, idx = val[:, :K], idx[:, :K]
    p, t = idx // V, idx % V
    d = (t == eos) & (eos >= 0)
    if done is not None:
        d = d | done.cpu().bool().view(N, W).gather(1, p)
    return val, p.int(), t.int(), d.to(torch.uint8)


def check(qg, logits, scores, N, W, K, done=None, eos=-1):
    got, ref = select(qg, logits, scores, N, W, K, done, eos), ref_select(logits, scores, N, W, K, done, eos)
    assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2]), (got[1], ref[1], got[2], ref[2])
    assert torch.equal(got[3], ref[3])
    # f32 sums of exponentials, in units of 2^-24: a thread's 16 values of a chunk in four sums (4 + 2), at
    # most 19 chunks here, 5 + 16 partials; the exponential 4; its argument 1.5 log2(e) E[max - x]
    # (mean under the distribution, 5 for these logits): 61.  Then the result's own rounding.
    fin = torch.isfinite(ref[0])
    assert torch.equal(fin, torch.isfinite(got[0]))
    err = (got[0].double() - ref[0]).abs()[fin]
    assert (err <= 64 * 2.0 ** -24 + 2.0 ** -24 * ref[0].abs()[fin]).all(), err.max()


def rand(N, W, V, seed=0, scale=2.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((N * W, V), generator=g) * scale).cuda(), (-20 * torch.rand((N * W,), generator=g)).cuda()


@pytest.mark.parametrize("V", [1, 2, 7, 63, 256, 1000, 2047, 2048, 2049, 8191, 8193, 32003, 151936])
@pytest.mark.parametrize("N,W,K", [(1, 1, 1), (1, 4, 4), (3, 5, 10)])
def test_sizes(qg, V, N, W, K):
    x, s = rand(N, W, V, seed=V)
    check(qg, x, s, N, W, min(K, W * V))


@pytest.mark.parametrize("K", [1, 17, 33, 64])
def test_many_picks(qg, K):
    x, s = rand(2, 6, 5000, seed=K)
    check(qg, x, s, 2, 6, K)


def test_large_batches(qg):
    x, s = rand(40, 8, 151936, seed=3)
    check(qg, x, s, 40, 8, 8)


def test_many_beams(qg):
    x, s = rand(2, 64, 3000, seed=4)
    check(qg, x, s, 2, 64, 64)


def test_a_pick_from_one_slice_or_beam(qg):
    """All picks from one beam and one slice: no part keeps fewer than K."""
    x, s = rand(1, 4, 20000, seed=5)
    x[2, 7000:7016] += 100
    check(qg, x, s, 1, 4, 16)
    s[:] = torch.tensor([-500.0, -1.0, -500.0, -500.0])
    check(qg, x, s, 1, 4, 16)


@pytest.mark.parametrize("V", [10, 3000, 70000])
def test_ties_go_to_the_lowest(qg, V):
    """Equal logits everywhere, equal beams, few distinct values, both zeros."""
    g = torch.Generator().manual_seed(6)
    for x in (torch.zeros((6, V)), torch.randint(-2, 2, (6, V), generator=g).float(),
              torch.where(torch.rand((6, V), generator=g) < 0.5, 0.0, -0.0)):
        x[3:] = x[:3]
        check(qg, x.cuda(), torch.full((6,), -2.0, device="cuda"), 2, 3, 7)


def test_banned_tokens(qg):
    """Rows almost wholly at -inf or the type's lowest value, fewer candidates than picks."""
    for low in (-math.inf, torch.finfo(torch.float32).min):
        x = torch.full((4, 9000), low)
        x[0, 5] = 1.0
        x[1, [8999, 17]] = torch.tensor([2.0, 2.5])
        x[3, 4000] = -3.0
        check(qg, x.cuda(), torch.tensor([-1.0, -2.0, -3.0, -4.0], device="cuda"), 1, 4, 8)


def test_rows_without_a_distribution(qg):
    """A row of -inf, one with +inf, NaN among values, a beam at -inf, and NaN as a score."""
    x, s = rand(1, 5, 700, seed=8)
    x[0] = -math.inf
    x[1, 30] = math.inf
    x[2, [0, 5, 699]] = math.nan
    s[3] = -math.inf
    check(qg, x, s, 1, 5, 10)
    s[2] = math.nan
    check(qg, x, s, 1, 5, 10)
    s[4] = math.inf
    check(qg, x, s, 1, 5, 10)
    check(qg, torch.full((2, 50), math.nan, device="cuda"), torch.zeros(2, device="cuda"), 1, 2, 9)


@pytest.mark.parametrize("eos", [0, 3, 4999])
def test_ended_beams(qg, eos):
    x, s = rand(3, 4, 5000, seed=9)
    done = torch.tensor([0, 1, 0, 0, 1, 1, 1, 1, 0, 0, 0, 0], dtype=torch.uint8, device="cuda")
    x[8, eos] = 30.0  # a live beam that ends now
    check(qg, x, s, 3, 4, 8, done, eos)
    check(qg, x, s, 3, 4, 8, done, -1)
    check(qg, x[:, :5].contiguous(), s, 3, 4, 12, done, min(eos, 4))


def test_unaligned_rows(qg):
    """A vocabulary that is no multiple of four, in a tensor that starts 4 bytes off."""
    x, s = rand(2, 3, 1001, seed=10)
    y = torch.empty(x.numel() + 1, device="cuda")[1:].view(6, 1001)
    y.copy_(x)
    check(qg, y, s, 2, 3, 6)


def test_neighbours_in_score(qg):
    """Candidates of different beams a few f32 steps apart are told apart in 64 bits."""
    V = 64
    x = torch.full((2, V), -8.0)
    x[0, 9], x[1, 4] = 3.0, 3.0
    s = torch.tensor([-7.0, -7.0])
    s[1] = torch.nextafter(s[1], torch.tensor(0.0))
    check(qg, x.cuda(), s.cuda(), 1, 2, 4)


def test_picks_feed_the_next_call(qg):
    """Two calls in a row on one workspace, on a side stream and in a graph."""
    N, W, K, V = 2, 4, 4, 4000
    x, s = rand(N, W, V, seed=11)
    want = select(qg, x, s, N, W, K)
    ws = torch.zeros(qg.beam_workspace_size(N, W, K, V), dtype=torch.uint8, device="cuda")
    o = [torch.zeros((N, K), device="cuda"), *[torch.zeros((N, K), dtype=torch.int32, device="cuda") for _ in range(2)]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg.beam_select(x, s, N, W, *o, ws)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.cpu(), b) for a, b in zip(o, want))
    st = torch.cuda.Stream()
    for t in o:
        t.zero_()
    torch.cuda.synchronize()
    qg.beam_select(x, s, N, W, *o, ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a.cpu(), b) for a, b in zip(o, want))


def test_shared_memory_of_an_earlier_kernel(qg):
    """The list of candidates starts empty whatever a kernel before left in its place: attention fills
    every SM's shared memory with a large pattern, the selection follows at once."""
    pat = torch.full((64, 64, 8, 128), 0x7BFF, dtype=torch.int16, device="cuda").view(torch.float16)
    cache = qg.kv_cache(pat, pat)
    lens = torch.full((4,), 1000, dtype=torch.int32, device="cuda")
    batch = qg.kv_batch(lens, torch.arange(64, dtype=torch.int32, device="cuda").view(4, 16))
    q = torch.zeros((4, 8, 128), dtype=torch.float16, device="cuda")
    out = torch.empty((4, 8, 128), device="cuda")
    aws = torch.empty(qg.attn_workspace_size(cache, batch, 8), dtype=torch.uint8, device="cuda")
    N, W, K, V = 8, 8, 8, 30000
    x, s = rand(N, W, V, seed=12)
    ref = ref_select(x, s, N, W, K)
    ws = torch.empty(qg.beam_workspace_size(N, W, K, V), dtype=torch.uint8, device="cuda")
    outs = [[torch.empty((N, K), device="cuda"), *[torch.empty((N, K), dtype=torch.int32, device="cuda") for _ in range(2)]]
            for _ in range(40)]
    for o in outs:
        qg.attn_paged(cache, batch, q, out, 0.1, aws)
        qg.beam_select(x, s, N, W, *o, ws)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[1].cpu(), ref[1]) and torch.equal(o[2].cpu(), ref[2])
