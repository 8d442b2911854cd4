"""Attention over the paged cache, through the C ABI, against a 64-bit reference: head layouts,
page sizes, ragged lengths, shared prefixes, rows that see nothing, strides, and what must not
be read.  The bound is kv_helpers.attention_tol."""
import pytest
import torch

from kv_helpers import DT, Batch, attention_ref, attention_tol, scale_of

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


def queries(T, Hq, D, dtype, seed=7, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, Hq, D), generator=g) * scale).to(DT[dtype]).cuda()


def attend(qg, bt, q, out_dtype, scale=None, plain_q=False, stream=None):
    T, Hq, D = q.shape
    cache, batch = qg.kv_cache(bt.k, bt.v), bt.desc(qg, plain_q)
    n = qg.attn_workspace_size(cache, batch, Hq)
    ws = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((T, Hq, D), float("nan"), dtype=out_dtype, device="cuda")
    torch.cuda.synchronize()
    qg.attn_paged(cache, batch, q, out, scale_of(D) if scale is None else scale, ws[:n], stream=stream)
    torch.cuda.synchronize()
    assert (ws[n:] == 0xA5).all(), "wrote past the workspace"
    return out


def check(qg, bt, Hq, dtype, out, seed=7, plain_q=False):
    q = queries(bt.T, Hq, bt.D, dtype, seed)
    out_dtype = torch.float32 if out == "f32" else DT[dtype]
    got = attend(qg, bt, q, out_dtype, plain_q=plain_q).double()
    ref, *terms = attention_ref(bt, q, scale_of(bt.D))
    assert torch.isfinite(got).all()
    err, tol = (got - ref).abs(), attention_tol(ref, *terms, bt.D, dtype, out_dtype)
    worst = (err / tol).max().item()
    assert worst <= 1.0, (worst, torch.nonzero(err > tol)[:4].tolist())
    assert qg.device_status() == 0
    return got


# (n, own, groups): new and own tokens per sequence, (first, end, prefix length) of each group
DECODE = {
    "one key": ([1], [1], ()),
    "seventeen": ([1], [17], ()),
    "long": ([1], [5003], ()),
    "ragged": ([1] * 7, [1, 2, 15, 16, 33, 700, 129], ()),
    "empty rows": ([1] * 5, [0, 3, 0, 40, 0], ()),
    "prefix": ([1] * 5, [1, 9, 64, 2, 31], ((0, 5, 333),)),
    "prefix of nothing": ([1] * 3, [5, 1, 20], ((0, 3, 0),)),
    "own of nothing": ([1] * 3, [0, 4, 0], ((0, 3, 50),)),
    "beams": ([1] * 9, [5] * 3 + [8] * 3 + [17] * 3, ((0, 3, 41), (3, 6, 7), (6, 9, 130))),
    "some in no group": ([1] * 5, [30, 2, 8, 19, 1], ((0, 3, 100),)),
}


@pytest.mark.parametrize("name", DECODE)
@pytest.mark.parametrize("dtype,out", [("f16", "f32"), ("bf16", "same"), ("bf16", "f32"), ("f16", "same")])
def test_one_token_per_sequence(qg, name, dtype, out):
    n, own, groups = DECODE[name]
    bt = Batch(n, own, 2, 128, 16, dtype, groups)
    check(qg, bt, 8, dtype, out, plain_q=True)


@pytest.mark.parametrize("Hkv,G", [(1, 1), (3, 1), (1, 5), (2, 7), (1, 16), (8, 4)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_layouts(qg, Hkv, G, D):
    bt = Batch([1, 1, 1], [70, 3, 200], Hkv, D, 32, "f16", ((1, 3, 37),), layout="hnd")
    check(qg, bt, Hkv * G, "f16", "f32")


@pytest.mark.parametrize("page", [1, 2, 8, 64, 1024])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_page_sizes(qg, page, layout):
    bt = Batch([1, 2, 1], [130, 17, 64], 2, 64, page, "bf16", ((0, 2, 45),), layout=layout)
    check(qg, bt, 4, "bf16", "same")


@pytest.mark.parametrize("page", [1, 2, 4, 8, 32, 64, 256])
@pytest.mark.parametrize("layout,D", [("nhd", 128), ("hnd", 64)])
def test_page_sizes_of_many_rows(qg, page, layout, D):
    """Enough rows for the tensor-core row tiles, lists that end inside a page and inside a key tile."""
    bt = Batch([70, 1, 33], [300, 9, 61], 2, D, page, "bf16", ((0, 2, 131), (2, 3, 256)), layout=layout)
    check(qg, bt, 8, "bf16", "f32")


QUERIES = {
    "two each": ([2, 2, 2], [2, 50, 9], ()),
    "ragged few": ([1, 3, 0, 5, 2], [40, 3, 12, 33, 2], ((0, 5, 77),)),
    "more queries than own tokens": ([4, 6], [2, 0], ((0, 1, 10),)),
    "around a row tile": ([31, 32, 33, 1], [31, 60, 33, 500], ()),
    "a prompt": ([300], [300], ()),
    "a prompt after tokens": ([257, 1, 40], [400, 90, 40], ()),
    "prompts under a prefix": ([130, 65, 1, 200], [130, 70, 6, 200], ((0, 4, 260),)),
    "prompts under prefixes": ([70, 33, 64], [70, 40, 129], ((0, 1, 128), (1, 3, 129))),
    "many short under a prefix": ([3] * 40, [3] * 40, ((0, 40, 600),)),
    "a prompt that sees little": ([150], [20], ((0, 1, 30),)),
    "short ones among prompts": ([1, 2, 90, 1, 1, 130, 3, 1, 140, 7], [9, 2, 90, 70, 1, 200, 3, 5, 141, 300],
                                 ((0, 7, 300), (7, 9, 77))),
    "whole and half tiles in turn": ([64, 33, 65, 40, 1, 129, 20, 64], [64, 333, 65, 300, 1, 400, 20, 900], ((0, 8, 140),)),
    "a short prefix before prompts": ([133, 129, 1], [133, 500, 40], ((0, 3, 5),)),
}


@pytest.mark.parametrize("name", QUERIES)
@pytest.mark.parametrize("dtype,out,D,G", [("f16", "f32", 128, 4), ("bf16", "same", 128, 4), ("bf16", "f32", 64, 5),
                                           ("f16", "same", 64, 8), ("bf16", "same", 256, 2), ("bf16", "same", 128, 1)])
def test_several_tokens_per_sequence(qg, name, dtype, out, D, G):
    n, own, groups = QUERIES[name]
    bt = Batch(n, own, 2, D, 16, dtype, groups)
    check(qg, bt, 2 * G, dtype, out)


def test_long_prefix_many_sequences(qg):
    """Rows enough for several row tiles over one long prefix, and own tails of every length."""
    B = 70
    bt = Batch([1] * B, [1 + (7 * i) % 45 for i in range(B)], 2, 128, 64, "bf16", ((0, B, 4099),))
    check(qg, bt, 16, "bf16", "same", plain_q=True)
    check(qg, bt, 16, "bf16", "f32", plain_q=True)


@pytest.mark.parametrize("big", [8.0, 40.0])
@pytest.mark.parametrize("n", [1, 150])
def test_peaked_scores(qg, big, n):
    """Scores hundreds apart, rising along the keys: the running maximum moves all the time."""
    bt = Batch([n], [600], 1, 128, 16, "f16", ())
    q = queries(bt.T, 4, 128, "f16", scale=big)
    order = torch.argsort(torch.einsum("sd,d->s", bt.rows[0][0][:, 0].float(), q[-1, 0].float().cpu()))
    k = bt.rows[0][0][order]
    bt.rows[0][0] = k
    for s in range(600):
        bt.k[bt.pages[0, s // 16].item(), s % 16] = k[s].cuda()
    got = attend(qg, bt, q, torch.float32).double()
    ref, *terms = attention_ref(bt, q, scale_of(128))
    tol = attention_tol(ref, *terms, 128, "f16", torch.float32)
    assert ((got - ref).abs() <= tol).all(), ((got - ref).abs() / tol).max()


@pytest.mark.parametrize("scale", [-0.07, 0.0, 1e-3])
@pytest.mark.parametrize("n", [1, 100])
def test_any_scale(qg, scale, n):
    """A negative scale turns the order of the scores round, zero makes every weight equal."""
    bt = Batch([n, 1], [200 + n, 40], 2, 128, 16, "f16", ((0, 2, 60),))
    q = queries(bt.T, 8, 128, "f16")
    got = attend(qg, bt, q, torch.float32, scale=scale).double()
    ref, *terms = attention_ref(bt, q, scale)
    assert ((got - ref).abs() <= attention_tol(ref, *terms, 128, "f16", torch.float32)).all()


@pytest.mark.parametrize("n,G", [(1, 4), (3, 8)])
def test_hundreds_of_sequences(qg, n, G):
    """More segments than a block has threads, a few prompts among them, in three groups."""
    B = 330
    ns = [n] * B
    for b in (0, 100, 101, 329):
        ns[b] = 45
    own = [ns[b] + (11 * b) % 60 for b in range(B)]
    bt = Batch(ns, own, 1, 64, 8, "bf16", ((0, 90, 100), (90, 91, 17), (91, 320, 333)))
    check(qg, bt, G, "bf16", "f32")


@pytest.mark.parametrize("D", [64, 256])
def test_starts_that_do_not_rise_reach_nothing(qg, D):
    """Overlapping token ranges give segments more tokens than there are: reported, and the
    workspace's end is kept (attend checks it)."""
    bt = Batch([60] * 12, [100] * 12, 2, D, 16, "f16", ((0, 6, 50), (6, 12, 50)), stale=0.0)
    q = queries(bt.T, 32, D, "f16")
    bt.q_start = torch.tensor([0, 720] * 6 + [0], dtype=torch.int32, device="cuda")
    attend(qg, bt, q, torch.float32)
    bt.q_start = torch.tensor([720, -5] * 6 + [1 << 30], dtype=torch.int32, device="cuda")
    bt.group_start = torch.tensor([9, -3, 1 << 30], dtype=torch.int32, device="cuda")
    attend(qg, bt, q, torch.float32)
    qg.device_status()


@pytest.mark.parametrize("n", [1, 64])
def test_infinite_scores_of_masked_keys(qg, n):
    """Keys past the length hold infinities and NaN, in the page's tail and in unused pages; the
    same call with finite garbage gives the same bits."""
    outs = []
    for stale in (float("nan"), float("inf"), 0.25):
        bt = Batch([n], [n + 5], 2, 128, 16, "f16", ((0, 1, 21),), stale=stale)
        outs.append(attend(qg, bt, queries(bt.T, 8, 128, "f16"), torch.float32))
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])


def test_rows_of_a_wider_tensor(qg):
    bt = Batch([1, 4, 2], [40, 9, 120], 2, 128, 16, "bf16", ())
    q = queries(bt.T, 8, 128, "bf16")
    wide = torch.full((bt.T, 3 * 8 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1024:2048] = q.view(bt.T, -1)
    got = attend(qg, bt, wide[:, 1024:2048].unflatten(1, (8, 128)), torch.bfloat16)
    assert torch.equal(got, attend(qg, bt, q, torch.bfloat16))


def test_repeats_are_bit_equal_and_need_no_clean_workspace(qg):
    bt = Batch([1] * 12, [300 + i for i in range(12)], 2, 128, 16, "bf16", ((0, 12, 900),))
    q = queries(bt.T, 16, 128, "bf16")
    a = attend(qg, bt, q, torch.float32)
    for _ in range(3):
        assert torch.equal(a, attend(qg, bt, q, torch.float32))


def test_far_pages_of_a_large_pool(qg):
    """Offsets past 2^32 bytes and 2^31 elements: the pages used lie at the end of a 5 GB pool."""
    Hkv, D, page = 8, 128, 16
    total = (5 << 30) // (page * Hkv * D * 2)
    k, v = (torch.empty((total, page, Hkv, D), dtype=torch.float16, device="cuda") for _ in range(2))
    bt = Batch([1, 40], [50, 61], Hkv, D, page, "f16", ())
    used = bt.k.shape[0]
    k[-used:], v[-used:] = bt.k, bt.v
    q = queries(bt.T, 32, D, "f16")
    want = attend(qg, bt, q, torch.float32)
    bt.k, bt.v = k, v
    bt.pages = torch.where(bt.pages >= 0, bt.pages + (total - used), bt.pages)
    assert torch.equal(want, attend(qg, bt, q, torch.float32))


@pytest.mark.parametrize("n", [1, 40])
def test_bad_pages_and_lengths_set_the_status(qg, n):
    """Page ids outside the pool and lengths past the page list are reported and reach nothing."""
    for what in ("page", "low page", "length", "negative"):
        bt = Batch([n, n], [60, 60], 2, 64, 16, "f16", (), stale=0.0, extra_cols=0)
        if what == "page":
            bt.pages[0, 1] = bt.k.shape[0]
        elif what == "low page":
            bt.pages[0, 0] = -1
        elif what == "length":
            bt.kv_len[0] = 1 << 30
            bt.pages[bt.pages < 0] = 0
        else:
            bt.kv_len[0] = -5
        q = queries(bt.T, 4, 64, "f16")
        out = attend(qg, bt, q, torch.float32)
        assert qg.device_status() == 1 << qg.QG_EDEVICE_ID, what
        bt.own[0] = 0
        ref, *terms = attention_ref(bt, q, scale_of(64))
        ok = (out.double() - ref).abs() <= attention_tol(ref, *terms, 64, "f16", torch.float32)
        assert ok[n:].all(), what  # the other sequence is untouched
        if what == "negative":
            assert not out[:n].any()


def test_on_a_side_stream_and_in_a_graph(qg):
    bt = Batch([1] * 6, [20, 300, 4, 70, 1, 9], 2, 128, 16, "bf16", ((0, 6, 200),))
    q = queries(bt.T, 8, 128, "bf16")
    want = attend(qg, bt, q, torch.bfloat16)
    s = torch.cuda.Stream()
    assert torch.equal(want, attend(qg, bt, q, torch.bfloat16, stream=s))
    cache, batch = qg.kv_cache(bt.k, bt.v), bt.desc(qg)
    ws = torch.zeros(qg.attn_workspace_size(cache, batch, 8), dtype=torch.uint8, device="cuda")
    out = torch.zeros((bt.T, 8, 128), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg.attn_paged(cache, batch, q, out, scale_of(128), ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, out)
    # the lengths are read when the graph runs
    bt.kv_len.copy_(torch.tensor([20, 299, 4, 70, 1, 9], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and not torch.equal(out[1], want[1])


def test_no_tokens(qg):
    bt = Batch([0, 0], [5, 9], 2, 64, 16, "f16", ())
    q = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    cache, batch = qg.kv_cache(bt.k, bt.v), bt.desc(qg)
    ws = torch.zeros(max(16, qg.attn_workspace_size(cache, batch, 4)), dtype=torch.uint8, device="cuda")
    qg.attn_paged(cache, batch, q, torch.empty((0, 4, 64), device="cuda"), 1.0, ws)
    torch.cuda.synchronize()
    assert qg.device_status() == 0


def test_pieces_of_tens_of_millions_of_keys(qg):
    """A worker's piece may take longer than a quarter of a second: no role gives up on another that is at
    work.  One page again and again, so 50 million keys need 16 MB; every value is 1."""
    T, D, G, keys = 2 * 152 * 16, 64, 16, 48 << 20
    k = torch.randn((1, 65536, 1, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    v = torch.ones_like(k)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = qg.kv_batch(i32([keys]), torch.zeros((1, keys >> 16), dtype=torch.int32, device="cuda"), i32([0, T]), T)
    cache = qg.kv_cache(k, v)
    q = queries(T, G, D, "bf16")
    out = torch.zeros((T, G, D), device="cuda")
    ws = torch.empty(qg.attn_workspace_size(cache, batch, G), dtype=torch.uint8, device="cuda")
    qg.attn_paged(cache, batch, q, out, scale_of(D), ws)
    torch.cuda.synchronize()
    assert qg.device_status() == 0
    # sums of cnt / 16 + 32 additions within 2^-23, in numerator and denominator alike
    assert ((out - 1).abs() <= 2 * (keys / 16 + 32) * 2.0 ** -23).all()
