"""Host checks of the drafted-decode calls: every refusal comes back before anything is enqueued (without a GPU a
launch attempt would return QG_ECUDA instead)."""
import ctypes
import math

import pytest

SHAPE, PTR, ALIGN, UNSUP, WS = 1, 2, 3, 4, 8
A, ODD = 1 << 20, (1 << 20) + 2


@pytest.fixture(scope="module")
def qg():
    import gguf_block_dequant_gb300 as qg
    from gguf_block_dequant_gb300 import build

    build.build()
    qg.load()
    return qg


def delta(qg, ws=A, n=1 << 50, **kw):
    g = dict(n_seqs=3, n_tokens=3, max_new=0, Hk=2, Hv=4, Dk=128, Dv=128, head_order=0, l2norm=1, n_slots=8, eps=1e-6, scale=0.1,
             q=A, k=A, v=A, a=A, b=A, q_stride=256, k_stride=256, v_stride=512, a_stride=4, b_stride=4, states=A,
             slot_stride=4 * 128 * 128, state_in=A, state_out=A, out=A, out_stride=512)
    g.update(kw)
    return qg.load().qg_delta_rule(ctypes.byref(qg.DeltaArgs(**g)), ws, n, None)


def test_delta_arguments(qg):
    for kw, want in [
        (dict(n_seqs=-1), SHAPE), (dict(n_seqs=70000), SHAPE), (dict(n_tokens=-1), SHAPE), (dict(n_tokens=1 << 25, q_start=A), SHAPE),
        (dict(n_tokens=4), SHAPE), (dict(max_new=-1), SHAPE), (dict(Hk=0), SHAPE), (dict(Hv=1), SHAPE), (dict(Hv=5), SHAPE),
        (dict(Hk=1025, Hv=1025), SHAPE), (dict(Dk=96), UNSUP), (dict(Dk=256), UNSUP), (dict(Dv=48), UNSUP), (dict(Dv=0), UNSUP),
        (dict(Dv=1056), UNSUP), (dict(head_order=2), SHAPE), (dict(l2norm=2), SHAPE), (dict(n_slots=-1), SHAPE),
        (dict(eps=-1.0), SHAPE), (dict(eps=math.nan), SHAPE), (dict(a_scale=A), PTR), (dict(a_bias=A), PTR),
        (dict(q_stride=252), SHAPE), (dict(k_stride=128), SHAPE), (dict(v_stride=0), SHAPE), (dict(out_stride=-512), SHAPE),
        (dict(a_stride=3), SHAPE), (dict(b_stride=1 << 40), SHAPE), (dict(slot_stride=4 * 128 * 128 - 4), SHAPE),
        (dict(q_stride=258), ALIGN), (dict(out_stride=513), ALIGN), (dict(slot_stride=4 * 128 * 128 + 2), ALIGN),
        (dict(q=A + 4), ALIGN), (dict(k=A + 8), ALIGN), (dict(v=ODD), ALIGN), (dict(out=A + 4), ALIGN), (dict(states=A + 8), ALIGN),
        (dict(a=ODD), ALIGN), (dict(b=ODD), ALIGN), (dict(a_scale=ODD, a_bias=A), ALIGN), (dict(q_start=ODD), ALIGN),
        (dict(state_in=ODD), ALIGN), (dict(state_out=ODD), ALIGN), (dict(state_each=ODD), ALIGN),
        (dict(q=None), PTR), (dict(k=None), PTR), (dict(v=None), PTR), (dict(a=None), PTR), (dict(b=None), PTR),
        (dict(out=None), PTR), (dict(states=None), PTR), (dict(n_slots=0), PTR),
        (dict(n_seqs=0, n_tokens=0), 0), (dict(n_tokens=0, q_start=A), 0),
    ]:
        assert delta(qg, **kw) == want, kw
    L = qg.load()
    assert L.qg_delta_rule(None, A, 1 << 40, None) == PTR
    assert L.qg_delta_workspace_size(None) == 0
    need = qg.delta_workspace_size(5000, 2, 2, 4, 128, 128)
    if need:
        long = dict(n_tokens=5000, n_seqs=2, q_start=A)
        assert delta(qg, ws=None, **long) == WS and delta(qg, n=need - 1, **long) == WS and delta(qg, ws=A + 8, **long) == ALIGN


def test_delta_workspace_grows(qg):
    """More tokens or sequences never need less; single tokens and short runs need none."""
    sizes = [qg.delta_workspace_size(T, n, 2, 4, 128, 128) for T, n in ((1, 1), (100, 1), (100, 4), (5000, 4), (5000, 64))]
    assert sizes == sorted(sizes)
    assert qg.delta_workspace_size(64, 64, 2, 4, 128, 128, 1) == 0
    assert qg.delta_workspace_size(100, 20, 2, 4, 128, 128, 7) == 0
    assert qg.delta_workspace_size(100, 20, 2, 4, 96, 128, 7) == 0  # refused


def test_probs_arguments(qg):
    f = lambda x=A, t=None, T=2, V=100, p=A: qg.load().qg_token_probs(x, t, T, V, p, None)  # noqa: E731
    for kw, want in [(dict(T=-1), SHAPE), (dict(T=65536), SHAPE), (dict(V=0), SHAPE), (dict(V=(1 << 20) + 1), SHAPE), (dict(x=None), PTR),
                     (dict(p=None), PTR), (dict(x=A + 4), ALIGN), (dict(p=A + 8), ALIGN), (dict(t=ODD), ALIGN), (dict(T=0), 0)]:
        assert f(**kw) == want, kw


def test_verify_arguments(qg):
    def f(p=A, q=A, tok=A, u=A, un=A, qs=A, n=3, T=7, V=100, acc=A, nxt=A, kv=A, kept=A):
        return qg.load().qg_draft_verify(p, q, tok, u, un, qs, n, T, V, acc, nxt, kv, kept, None)

    for kw, want in [
        (dict(n=-1), SHAPE), (dict(n=65536), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 25), SHAPE), (dict(V=0), SHAPE),
        (dict(V=1 << 21), SHAPE), (dict(qs=None), SHAPE), (dict(p=None), PTR), (dict(tok=None), PTR), (dict(u=None), PTR),
        (dict(un=None), PTR), (dict(acc=None), PTR), (dict(nxt=None), PTR), (dict(kv=None), PTR), (dict(kept=None), PTR),
        (dict(p=A + 4), ALIGN), (dict(q=A + 8), ALIGN), (dict(tok=ODD), ALIGN), (dict(u=ODD), ALIGN), (dict(un=ODD), ALIGN),
        (dict(qs=ODD), ALIGN), (dict(acc=ODD), ALIGN), (dict(nxt=ODD), ALIGN), (dict(kv=ODD), ALIGN), (dict(kept=ODD), ALIGN),
        (dict(n=0, T=0), 0),
    ]:
        assert f(**kw) == want, kw


def cache(qg, **kw):
    c = dict(k=A, v=A, dtype=1, n_pages=8, page_size=16, n_heads=2, head_dim=128, page_stride=16 * 256, token_stride=256,
             head_stride=128)
    c.update(kw)
    return qg.KVCache(*[c[f] for f, _ in qg.KVCache._fields_])


def batch(qg, **kw):
    b = dict(n_seqs=3, n_tokens=0, n_groups=0, max_pages=4, max_prefix_pages=0, q_start=None, kv_len=A, pages=A,
             group_start=None, prefix_len=None, prefix_pages=None)
    b.update(kw)
    return qg.KVBatch(*[b[f] for f, _ in qg.KVBatch._fields_])


def test_page_call_arguments(qg):
    L = qg.load()
    two = lambda **kw: (qg.KVCache * 2)(cache(qg), cache(qg, **kw))  # noqa: E731
    ref = ctypes.byref

    def fork(c=None, b=None, refs=A, src=A, keep=A):
        return L.qg_kv_fork(ref(c or cache(qg)), ref(b or batch(qg)), refs, src, keep, None)

    def reserve(c=None, n=2, b=None, refs=A, add=A, miss=A, ws=A, size=1 << 40):
        return L.qg_kv_reserve(c or two(), n, ref(b or batch(qg)), refs, add, miss, ws, size, None)

    def compact(c=None, n=2, b=None, src=A, start=A, keep=A, k=5):
        return L.qg_kv_compact(c or two(), n, ref(b or batch(qg)), src, start, keep, k, None)

    for f in (fork, reserve, compact):
        for kw, want in [(dict(n_seqs=-1), SHAPE), (dict(n_seqs=70000), SHAPE), (dict(max_pages=0), SHAPE), (dict(kv_len=None), PTR),
                         (dict(pages=None), PTR), (dict(kv_len=ODD), ALIGN), (dict(pages=ODD), ALIGN), (dict(n_seqs=0), 0)]:
            assert f(b=batch(qg, **kw)) == want, (f, kw)
    for kw, want in [(dict(refs=None), PTR), (dict(refs=ODD), ALIGN), (dict(src=ODD), ALIGN), (dict(keep=ODD), ALIGN),
                     (dict(c=cache(qg, page_size=24)), SHAPE), (dict(c=cache(qg, k=None)), PTR), (dict(c=cache(qg, dtype=0)), UNSUP)]:
        assert fork(**kw) == want, kw
    need = L.qg_kv_reserve_workspace_size(two(), ref(batch(qg)))
    assert need > 0
    for kw, want in [(dict(refs=None), PTR), (dict(add=None), PTR), (dict(miss=None), PTR), (dict(refs=ODD), ALIGN), (dict(add=ODD), ALIGN),
                     (dict(miss=ODD), ALIGN), (dict(ws=None), WS), (dict(size=need - 1), WS), (dict(ws=A + 8), ALIGN),
                     (dict(n=0), SHAPE), (dict(n=129), SHAPE), (dict(c=two(n_pages=9)), SHAPE), (dict(c=two(dtype=2)), SHAPE),
                     (dict(c=two(v=None)), PTR)]:
        assert reserve(**kw) == want, kw
    for kw, want in [(dict(src=None), PTR), (dict(start=None), PTR), (dict(keep=None), PTR), (dict(src=ODD), ALIGN), (dict(start=ODD), ALIGN),
                     (dict(keep=ODD), ALIGN), (dict(k=-1), SHAPE), (dict(k=1 << 25), SHAPE), (dict(k=0), 0), (dict(n=0), SHAPE),
                     (dict(c=two(token_stride=512)), SHAPE)]:
        assert compact(**kw) == want, kw
    assert L.qg_kv_fork(None, ref(batch(qg)), A, A, A, None) == PTR
    assert L.qg_kv_fork(ref(cache(qg)), None, A, A, A, None) == PTR
    assert L.qg_kv_reserve_workspace_size(None, ref(batch(qg))) == 0


def test_binding_refuses_types_shapes_and_host_tensors(qg):
    torch = pytest.importorskip("torch")
    f, i = (lambda *s: torch.zeros(s)), (lambda *s: torch.zeros(s, dtype=torch.int32))  # noqa: E731
    good = dict(q=f(3, 2, 64), k=f(3, 2, 64), v=f(3, 4, 32), a=f(3, 4), b=f(3, 4), states=f(5, 4, 64, 32), state_in=i(3),
                state_out=i(3), out=f(3, 4, 32), stream=0)
    for kw in (dict(q=f(3, 128)), dict(k=f(3, 2, 32)), dict(k=f(3, 2, 64).half()), dict(v=f(2, 4, 32)), dict(a=f(3, 3)), dict(b=f(4, 4)),
               dict(b=f(3, 4).double()), dict(states=f(5, 4, 32, 64)), dict(states=f(5, 4, 64, 32).double()),
               dict(states=f(5, 4, 32, 64).transpose(2, 3)), dict(state_in=i(2)), dict(state_in=i(3).long()), dict(state_out=i(4)),
               dict(state_each=i(2)), dict(out=f(3, 4, 64)), dict(out=f(3, 32, 4).transpose(1, 2)), dict(q_start=i(4).long()),
               dict(q_start=i(3)), dict(a_scale=f(3), a_bias=f(4)), dict(a_scale=f(4), a_bias=f(4).half()), {}):
        with pytest.raises(ValueError):  # the last one: all as it should be, but not on a GPU
            qg.delta_rule(**{**good, **kw})
    for kw in (dict(logits=f(2, 9).half()), dict(probs=f(2, 8)), dict(temperature=f(3)), dict(temperature=i(2)),
               dict(logits=f(9, 2).T), {}):
        with pytest.raises(ValueError):
            qg.token_probs(**{**dict(logits=f(2, 9), probs=f(2, 9), stream=0), **kw})
    good = dict(probs=f(5, 9), tokens=i(5), u=f(5), u_next=f(2), accepted=i(2), next_token=i(2), q_start=i(3), stream=0)
    for kw in (dict(probs=f(9, 5).T), dict(tokens=i(4)), dict(tokens=f(5)), dict(u=f(4)), dict(u_next=f(3)), dict(accepted=i(3)),
               dict(next_token=i(2).long()), dict(draft_probs=f(4, 9)), dict(draft_probs=f(5, 9).half()), dict(kv_len=i(3)),
               dict(kept_len=f(2)), dict(q_start=None), {}):
        with pytest.raises(ValueError):
            qg.draft_verify(**{**good, **kw})
    k = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    cs, b = qg.kv_caches([k], [k.clone()]), qg.kv_batch(i(3), i(3, 5))
    for kw in (dict(refs=i(5)), dict(refs=f(4)), dict(src=i(2)), dict(keep=i(3).long()), {}):
        with pytest.raises(ValueError):
            qg.kv_fork(**{**dict(caches=cs, batch=b, refs=i(4), stream=0), **kw})
    for kw in (dict(refs=i(5)), dict(add=i(2)), dict(missing=i(2)), dict(add=f(3)), {}):
        with pytest.raises(ValueError):
            qg.kv_reserve(**{**dict(caches=cs, batch=b, refs=i(4), add=i(3), missing=i(1), workspace=i(999), stream=0), **kw})
    for kw in (dict(src=i(2)), dict(keep_start=i(3)), dict(keep=f(9)), {}):
        with pytest.raises(ValueError):
            qg.kv_compact(**{**dict(caches=cs, batch=b, src=i(3), keep_start=i(4), keep=i(9), stream=0), **kw})
