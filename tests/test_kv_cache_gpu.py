"""The paged cache's writers against 64-bit references: kv_append (norm, rotation, page writes)
and beam_reorder (page lists and part-filled pages, in place)."""
import pytest
import torch

from kv_helpers import DT, Batch, rope_ref

pytestmark = pytest.mark.gpu
THETA = 1000000.0


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


def append(qg, bt, Hq, dtype, rot, pairs, norm, seed=3, theta=THETA, plain_q=False, eps=1e-6, fused=True, stream=None,
           factors=None):
    """Runs kv_append on random rows; returns what went in and q_out."""
    D, Hkv, T = bt.D, bt.Hkv, bt.T
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, (Hq + 2 * Hkv) * D), generator=g) * 1.7).cuda()
    a, b = Hq * D, (Hq + Hkv) * D
    q, k, v = x[:, :a], x[:, a:b], x[:, b:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    wq = wk = None
    if norm:
        wq, wk = ((1 + 0.3 * torch.randn((D,), generator=g)).cuda() for _ in range(2))
    q_out = torch.full((T, Hq, D), float("nan"), dtype=DT[dtype], device="cuda")
    fr = qg.rope_freqs(rot, theta, factors).cuda() if rot else None
    qg.kv_append(qg.kv_cache(bt.k, bt.v), bt.desc(qg, plain_q), q, k, v, q_out, fr, pairs=pairs, q_norm=wq, k_norm=wk,
                 eps=eps, stream=stream)
    torch.cuda.synchronize()
    return x, wq, wk, q_out


def positions(bt):
    pos, slot, seq = [], [], []
    for b, n in enumerate(bt.n):
        pre = bt.group(b)[1]
        for i in range(n):
            slot.append(bt.own[b] - n + i)
            pos.append(pre + slot[-1])
            seq.append(b)
    return torch.tensor(pos, device="cuda"), slot, seq


def close16(got, ref, mag, dtype, what):
    """One rounding to 16 bits (half a step of the value, 2^-25 near f16's zero) of an f32 result
    whose terms (|x| w s, twice for a rotation) carry the norm's sum and root (D/32 + 5 + 3
    roundings: 16), the angle's and sine's 3 and the two products' and sum's 3: 24 * 2^-24."""
    half = torch.finfo(DT[dtype]).eps / 2
    tol = half * ref.abs() + (1 + half) * 24 * 2.0 ** -24 * mag + (2.0 ** -25 if dtype == "f16" else 1e-38)
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (what, (err / tol).max().item())


def verify(bt, x, wq, wk, q_out, k0, v0, Hq, dtype, rot, pairs, theta=THETA, eps=1e-6):
    D, Hkv, T = bt.D, bt.Hkv, bt.T
    pos, slot, seq = positions(bt)
    h = x.double().view(T, Hq + 2 * Hkv, D)
    q, k, v = h[:, :Hq], h[:, Hq:Hq + Hkv], h[:, Hq + Hkv:]
    if wq is not None:
        q = q / torch.sqrt(q.square().mean(-1, keepdim=True) + eps) * wq.double()
        k = k / torch.sqrt(k.square().mean(-1, keepdim=True) + eps) * wk.double()
    rq, rk = rope_ref(q, pos, rot, theta, pairs), rope_ref(k, pos, rot, theta, pairs)
    # magnitude of the two terms of each output
    i = torch.arange(rot // 2, device="cuda")
    ia, ib = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)

    def mag(y):
        m = y.abs().clone()
        s = y[..., ia].abs() + y[..., ib].abs()
        m[..., ia], m[..., ib] = s, s
        return m

    close16(q_out, rq, mag(q), dtype, "q")
    want_k, want_v = k0.clone(), v0.clone()
    for t in range(T):
        p, r = bt.pages[seq[t], slot[t] // bt.page].item(), slot[t] % bt.page
        close16(bt.k[p, r], rk[t], mag(k)[t], dtype, "k")
        assert torch.equal(bt.v[p, r], v[t].to(DT[dtype])), "v"
        want_k[p, r], want_v[p, r] = bt.k[p, r], bt.v[p, r]
    # nothing else of the pools changed
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(want_k), bits(bt.k)) and torch.equal(bits(want_v), bits(bt.v))


CASES = [
    # Hq, Hkv, D, rot, pairs, norm, dtype, layout, page
    (8, 2, 128, 128, False, True, "f16", "nhd", 16),
    (8, 2, 128, 64, True, True, "bf16", "hnd", 8),
    (5, 1, 64, 64, False, False, "bf16", "nhd", 1),
    (6, 3, 64, 16, True, False, "f16", "nhd", 32),
    (4, 4, 256, 64, False, True, "f16", "hnd", 16),
    (16, 1, 256, 256, True, True, "bf16", "nhd", 64),
    (2, 2, 64, 8, False, True, "f16", "nhd", 16),
    (2, 2, 128, 0, False, True, "f16", "nhd", 16),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("fused", [True, False])
def test_append(qg, case, fused):
    Hq, Hkv, D, rot, pairs, norm, dtype, layout, page = case
    bt = Batch([3, 1, 0, 20, 1], [3, 40, 7, 77, 1], Hkv, D, page, dtype, ((0, 3, 29),), layout=layout, stale=0.5)
    k0, v0 = bt.k.clone(), bt.v.clone()
    x, wq, wk, q_out = append(qg, bt, Hq, dtype, rot, pairs, norm, fused=fused)
    verify(bt, x, wq, wk, q_out, k0, v0, Hq, dtype, rot, pairs)
    assert qg.device_status() == 0


@pytest.mark.parametrize("B", [1, 9, 400])
def test_append_one_token_each(qg, B):
    bt = Batch([1] * B, [1 + (5 * i) % 37 for i in range(B)], 2, 128, 16, "f16", (), stale=0.0)
    k0, v0 = bt.k.clone(), bt.v.clone()
    x, wq, wk, q_out = append(qg, bt, 8, "f16", 128, False, True, plain_q=True)
    verify(bt, x, wq, wk, q_out, k0, v0, 8, "f16", 128, False)


@pytest.mark.parametrize("far", [131071, 1 << 24, (1 << 31) - 100])
def test_far_positions(qg, far):
    """Angles of far positions keep their accuracy: no f32 product of position and frequency."""
    bt = Batch([2, 1], [5, 60], 2, 128, 16, "f16", ((0, 2, 16),), stale=0.0)
    bt.groups = [(0, 2, far)]
    bt.prefix_len.fill_(far)
    k0, v0 = bt.k.clone(), bt.v.clone()
    x, wq, wk, q_out = append(qg, bt, 4, "f16", 128, False, False, theta=10000.0)
    verify(bt, x, wq, wk, q_out, k0, v0, 4, "f16", 128, False, theta=10000.0)


def test_frequency_factors(qg):
    """Factors divide the frequencies (the GGUF rope_freqs tensor)."""
    f = [1.0 + i / 7 for i in range(32)]
    a, b = qg.rope_freqs(64, 10000.0, f), qg.rope_freqs(64, 10000.0)
    got = (a.double() % 2.0 ** 64) / (b.double() % 2.0 ** 64)
    want = 1 / torch.tensor(f, dtype=torch.float32).double()
    # each entry is rounded to whole units, and its double before that
    unit = 0.5 / (a.double() % 2.0 ** 64) + 0.5 / (b.double() % 2.0 ** 64)
    assert ((got - want).abs() <= 2.0 ** -50 + want * unit).all()


def test_append_values_that_stay(qg):
    """Elements past the rotated part pass through untouched: infinities next to finite values."""
    bt = Batch([1], [1], 1, 64, 16, "bf16", (), stale=0.0)
    x = torch.ones((1, 3 * 64), device="cuda")
    x[0, 32], x[0, 64 + 40] = float("inf"), float("-inf")
    q_out = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    qg.kv_append(qg.kv_cache(bt.k, bt.v), bt.desc(qg), x[:, :64], x[:, 64:128], x[:, 128:], q_out,
                 qg.rope_freqs(32, THETA).cuda())
    torch.cuda.synchronize()
    want = x.view(3, 64).to(torch.bfloat16)  # position 0: the rotation is the identity
    p = bt.pages[0, 0].item()
    assert torch.equal(q_out[0, 0], want[0]) and torch.equal(bt.k[p, 0, 0], want[1]) and torch.equal(bt.v[p, 0, 0], want[2])


def test_append_bad_slots_set_the_status(qg):
    for what in ("page", "length", "no slot"):
        bt = Batch([1, 1], [20, 20], 1, 64, 16, "f16", (), stale=0.0, extra_cols=0)
        k0 = bt.k.clone()
        if what == "page":
            bt.pages[0, 1] = bt.k.shape[0]
        elif what == "length":
            bt.kv_len[0] = 33
        else:
            bt.kv_len[0] = 0
        x, *_, q_out = append(qg, bt, 2, "f16", 64, False, False)
        assert qg.device_status() == 1 << qg.QG_EDEVICE_ID, what
        p, r = bt.pages[1, 1].item(), 19 % 16
        assert torch.equal(bt.v[p, r, 0], x[1, -64:].half())  # the other sequence is written
        k0[p, r] = bt.k[p, r]
        assert torch.equal(k0, bt.k), what
        assert torch.isfinite(q_out).all()


def test_append_keys_only_on_a_side_stream(qg):
    bt = Batch([2, 1], [2, 30], 2, 64, 16, "bf16", (), stale=0.0)
    k0, v0 = bt.k.clone(), bt.v.clone()
    s = torch.cuda.Stream()
    g = torch.Generator().manual_seed(1)
    kv = torch.randn((bt.T, 4 * 64), generator=g).cuda()
    torch.cuda.synchronize()
    qg.kv_append(qg.kv_cache(bt.k, bt.v), bt.desc(qg), None, kv[:, :128], kv[:, 128:], None,
                 qg.rope_freqs(64, THETA).cuda(), stream=s)
    torch.cuda.synchronize()
    x = torch.cat([torch.zeros((bt.T, 128), device="cuda"), kv], 1)
    verify(bt, x, None, None, torch.zeros((bt.T, 2, 64), dtype=torch.bfloat16, device="cuda"), k0, v0, 2, "bf16", 64,
           False)


# ---- beam_reorder -------------------------------------------------------------------------------

def reorder_case(N, W, lens, page, Hkv=2, D=64, layers=3, dtype="f16", layout="nhd", seed=0, cols=None):
    g = torch.Generator().manual_seed(seed)
    cols = cols or max(lens) // page + 1
    total = N * W * cols + 2
    dims = (page, Hkv, D) if layout == "nhd" else (Hkv, page, D)
    pool = torch.randn((2 * layers, total, *dims), generator=g).to(DT[dtype]).cuda()
    if layout == "hnd":
        pool = pool.permute(0, 1, 3, 2, 4)
    pages = torch.randperm(total, generator=g)[:N * W * cols].view(N * W, cols).to(torch.int32).cuda()
    kv_len = torch.tensor([x for x in lens for _ in range(W)], dtype=torch.int32).cuda()
    return pool, pages, kv_len


def tokens_of(pool, pages, b, n, page):
    return torch.stack([pool[:, pages[b, s // page].item(), s % page] for s in range(n)]) if n else None


def run_reorder(qg, pool, pages, kv_len, parents, W):
    caches = qg.kv_caches(list(pool[0::2]), list(pool[1::2]))
    qg.beam_reorder(caches, qg.kv_batch(kv_len, pages), parents, W)
    torch.cuda.synchronize()


@pytest.mark.parametrize("W", [2, 3, 5, 9, 16, 17, 32])
@pytest.mark.parametrize("page,lens", [(16, [37, 16, 5]), (8, [0, 8, 15]), (1, [3, 1, 2]), (64, [63, 130, 64])])
def test_reorder_gives_each_beam_its_parents_tokens(qg, W, page, lens):
    """Every beam's tokens become its parent's, whatever the parents: cycles, one parent for all."""
    g = torch.Generator().manual_seed(W)
    layout = "hnd" if W % 2 else "nhd"
    for how in ("random", "cycle", "all of one", "same"):
        pool, pages, kv_len = reorder_case(len(lens), W, lens, page, layout=layout)
        par = {"random": torch.randint(0, W, (len(lens), W), generator=g),
               "cycle": ((torch.arange(W) + 1) % W).expand(len(lens), W),
               "all of one": torch.full((len(lens), W), W - 1),
               "same": torch.arange(W).expand(len(lens), W)}[how].to(torch.int32).contiguous().cuda()
        before, own = pool.clone(), pages.clone()
        want = [tokens_of(pool, pages, r * W + par[r, i].item(), lens[r], page)
                for r in range(len(lens)) for i in range(W)]
        run_reorder(qg, pool, pages, kv_len, par, W)
        for b in range(len(lens) * W):
            got = tokens_of(pool, pages, b, lens[b // W], page)
            assert (got is None and want[b] is None) or torch.equal(got, want[b]), (how, b)
            full = lens[b // W] // page
            assert torch.equal(pages[b, full:], own[b, full:])  # its own page keeps filling
        # full pages are shared, not copied
        for r in range(len(lens)):
            full = lens[r] // page
            if full:
                used = own[r * W:(r + 1) * W, :full].flatten().long()
                assert torch.equal(pool[:, used], before[:, used])
    assert qg.device_status() == 0


def test_reorder_refuses_unequal_beams_and_bad_parents(qg):
    W, page = 3, 8
    pool, pages, kv_len = reorder_case(2, W, [13, 10], page)
    kv_len[1] = 12  # request 0 is left as it is; request 1 moves
    par = torch.tensor([[1, 0, 2], [2, 7, 0]], dtype=torch.int32).cuda()
    before, own = pool.clone(), pages.clone()
    want = [tokens_of(pool, pages, 3 + p, 10, page) for p in (2, 1, 0)]  # a bad parent keeps its own state
    run_reorder(qg, pool, pages, kv_len, par, W)
    assert qg.device_status() == 1 << qg.QG_EDEVICE_ID
    assert torch.equal(pages[:3], own[:3]) and torch.equal(pool[:, own[:3].flatten().long()], before[:, own[:3].flatten().long()])
    for i in range(3):
        assert torch.equal(tokens_of(pool, pages, 3 + i, 10, page), want[i])


def test_reorder_bad_pages_and_lengths(qg):
    W, page = 2, 8
    for what in ("page", "length", "negative"):
        pool, pages, kv_len = reorder_case(1, W, [13], page)
        if what == "page":
            pages[1, 1] = pool.shape[1]
        else:
            kv_len.fill_(8 * pages.shape[1] + 1 if what == "length" else -3)
        before, own = pool.clone(), pages.clone()
        run_reorder(qg, pool, pages, kv_len, torch.tensor([[1, 0]], dtype=torch.int32).cuda(), W)
        assert qg.device_status() == 1 << qg.QG_EDEVICE_ID, what
        assert torch.equal(pool, before)
        if what != "page":
            assert torch.equal(pages, own)


def test_reorder_bad_page_leaves_the_lists_too(qg):
    """A bad page in the column being filled: no block of the request moves anything, the page lists'
    among them (full pages of one beam with the begun page of another would be a mixed history)."""
    W, page = 3, 8
    for lens in ([13, 21], [21, 13]):
        pool, pages, kv_len = reorder_case(2, W, lens, page)
        pages[1, lens[0] // page] = -1
        before, own = pool.clone(), pages.clone()
        par = torch.tensor([[1, 0, 2], [2, 0, 1]], dtype=torch.int32).cuda()
        want = [tokens_of(pool, pages, W + p, lens[1], page) for p in (2, 0, 1)]
        run_reorder(qg, pool, pages, kv_len, par, W)
        assert qg.device_status() == 1 << qg.QG_EDEVICE_ID
        assert torch.equal(pages[:W], own[:W])
        used = own[:W][own[:W] >= 0].long()
        assert torch.equal(pool[:, used], before[:, used])
        for i in range(W):  # the other request moves
            assert torch.equal(tokens_of(pool, pages, W + i, lens[1], page), want[i])


def test_frequency_factors_on_the_gpu(qg):
    """The table is made on the host: factors that lie on the GPU (a loaded rope_freqs tensor) come over first."""
    f = torch.linspace(1.0, 8.0, 32)
    assert torch.equal(qg.rope_freqs(64, 10000.0, f.cuda()), qg.rope_freqs(64, 10000.0, f))
    assert torch.equal(qg.rope_freqs(64, 10000.0, f.double().cuda()), qg.rope_freqs(64, 10000.0, f.tolist()))
