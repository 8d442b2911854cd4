"""NaN and infinities in attention over the paged cache: a NaN score makes its row NaN however the
row's keys were cut into pieces."""
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
