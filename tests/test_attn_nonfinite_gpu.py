"""NaN and infinities in attention over the paged cache: a NaN score makes its row NaN however the
row's keys were cut into pieces, and a value that a token must not see has no effect on it."""
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


def queries(T, Hq, D, dtype, seed=7):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, Hq, D), generator=g) * 2.0).to(DT[dtype]).cuda()


def attend(qg, bt, q, out_dtype):
    T, Hq, D = q.shape
    cache, batch = qg.kv_cache(bt.k, bt.v), bt.desc(qg)
    ws = torch.full((qg.attn_workspace_size(cache, batch, Hq),), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((T, Hq, D), 7.0, dtype=out_dtype, device="cuda")
    qg.attn_paged(cache, batch, q, out, scale_of(D), ws)
    torch.cuda.synchronize()
    assert qg.device_status() == 0
    return out


def place(bt, which, s):
    """Page and row of token s of a list (sequence b: b; group g: number of sequences + g)."""
    B = len(bt.n)
    table = bt.pages[which] if which < B else bt.prefix_pages[which - B]
    return table[s // bt.page].item(), s % bt.page


# (n, own, groups): rows in one piece and in many, of the kernel for few rows and of the one for many
SPLIT = {
    "few rows, one piece": ([1], [17], ()),
    "few rows, many pieces": ([1, 1], [5003, 40], ()),
    "few rows, prefix and own": ([1] * 3, [5, 1, 20], ((0, 3, 333),)),
    "many rows, one piece or two": ([150, 40], [150, 40], ()),
    "many rows, many pieces": ([20, 33], [4000, 900], ()),
    "many rows, prefix and own": ([70, 33, 64], [70, 40, 129], ((0, 1, 128), (1, 3, 600))),
    "a decode step under a prefix": ([1] * 40, [1 + i for i in range(40)], ((0, 40, 3000),)),
}


def compare(got, ref, terms, D, dtype, out_dtype):
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), "NaN in the wrong rows"
    tol = attention_tol(ref, *terms, D, dtype, out_dtype)
    err = (got.double() - ref).abs()
    assert ((err <= tol) | torch.isnan(ref)).all()


@pytest.mark.parametrize("name", SPLIT)
@pytest.mark.parametrize("dtype,out,D,G", [("f16", "f32", 128, 4), ("bf16", "same", 64, 8), ("bf16", "f32", 256, 2)])
def test_nan_in_a_query(qg, name, dtype, out, D, G):
    n, own, groups = SPLIT[name]
    bt = Batch(n, own, 2, D, 16, dtype, groups)
    q = queries(bt.T, 2 * G, D, dtype)
    q[0, 1, 3] = q[bt.T - 1, 2 * G - 1, 0] = float("nan")
    out_dtype = torch.float32 if out == "f32" else DT[dtype]
    ref, *terms = attention_ref(bt, q, scale_of(D))
    assert torch.isnan(ref[0, 1]).all() and torch.isnan(ref[-1, -1]).all()
    compare(attend(qg, bt, q, out_dtype), ref, terms, D, dtype, out_dtype)


@pytest.mark.parametrize("name", SPLIT)
@pytest.mark.parametrize("dtype,out,D,G", [("f16", "f32", 128, 4), ("bf16", "same", 64, 8), ("bf16", "f32", 256, 2)])
def test_nan_in_a_run_of_keys(qg, name, dtype, out, D, G):
    """Keys that fill a piece (or all of a list): the tokens that see them are NaN, the others
    untouched."""
    n, own, groups = SPLIT[name]
    for which in range(len(n) + len(groups)):
        ln = own[which] if which < len(n) else groups[which - len(n)][2]
        bt = Batch(n, own, 2, D, 16, dtype, groups)
        for s in range(ln // 3, min(ln, ln // 3 + 300)):
            bt.rows[which][0][s, 0] = float("nan")  # of the first cached head
            bt.k[(*place(bt, which, s), 0)] = float("nan")
        q = queries(bt.T, 2 * G, D, dtype)
        out_dtype = torch.float32 if out == "f32" else DT[dtype]
        ref, *terms = attention_ref(bt, q, scale_of(D))
        assert torch.isnan(ref).any() and not torch.isnan(ref[:, G:]).any()
        compare(attend(qg, bt, q, out_dtype), ref, terms, D, dtype, out_dtype)
        if which >= 3:
            break


MASKED = {
    "a draft": ([3], [40], ()),
    "drafts under a prefix": ([1, 3, 2, 4], [9, 30, 2, 64], ((0, 4, 77),)),
    "more queries than tokens": ([4, 6], [2, 0], ((0, 1, 10),)),
    "half a row tile": ([20], [300], ()),
    "a prompt": ([300], [300], ()),
    "prompts of every kind": ([130, 65, 1, 20], [130, 70, 6, 200], ((0, 4, 260),)),
    "a prompt that sees little": ([150], [20], ((0, 1, 30),)),
    "short ones of which some see little": ([3] * 40, [3 if i % 2 else 1 for i in range(40)], ((0, 40, 6),)),
}


@pytest.mark.parametrize("name", MASKED)
@pytest.mark.parametrize("dtype,out,D,G", [("f16", "f32", 128, 4), ("bf16", "same", 128, 8), ("bf16", "f32", 64, 5),
                                           ("f16", "same", 256, 2), ("bf16", "f32", 128, 1)])
def test_values_a_token_must_not_see(qg, name, dtype, out, D, G):
    """Infinite and NaN values of tokens past a token's own: its output keeps its bits.  Tokens that see
    one have no finite output in that element, and the same bits in all others."""
    n, own, groups = MASKED[name]
    out_dtype = torch.float32 if out == "f32" else DT[dtype]
    bt = Batch(n, own, 2, D, 16, dtype, groups)
    q = queries(bt.T, 2 * G, D, dtype)
    want = attend(qg, bt, q, out_dtype)
    assert torch.isfinite(want).all()
    hit = torch.zeros((bt.T, 2 * G, D), dtype=torch.bool)
    vals = [float("inf"), float("-inf"), float("nan")]
    c = 0
    for which in range(len(n) + len(groups)):
        ln = own[which] if which < len(n) else groups[which - len(n)][2]
        last = range(max(0, ln - (n[which] if which < len(n) else 5)), ln)
        for s in [*last[:1], *last[len(last) // 2:len(last) // 2 + 1], *last[-1:]]:
            h, col = c % 2, (37 * c + 5) % D
            bt.v[(*place(bt, which, s), h, col)] = vals[c % 3]
            c += 1
            for b in range(len(n)):
                g, pre = bt.group(b)
                mine = which == b or (g >= 0 and which == len(n) + g)
                for i in range(n[b] if mine else 0):
                    seen = (own[b] if which == b else pre + own[b]) - n[b] + i + 1
                    if s < seen:
                        hit[bt.qs[b] + i, h * G:(h + 1) * G, col] = True
    got = attend(qg, bt, q, out_dtype)
    hit = hit.cuda()
    same = (got == want) | hit
    assert same.all(), torch.nonzero(~same)[:4].tolist()
    assert not torch.isfinite(got[hit]).any()
