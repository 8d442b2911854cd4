"""Host checks of the cached-decode calls: every refusal comes back before anything is enqueued
(without a GPU a launch attempt would return QG_ECUDA instead), and the rotation table."""
import ctypes
import math

import pytest

P, I, I64, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
SHAPE, PTR, ALIGN, UNSUP, WS = 1, 2, 3, 4, 8
A, ODD = 1 << 20, (1 << 20) + 2


@pytest.fixture(scope="module")
def qg():
    import gguf_block_dequant_gb300 as qg
    from gguf_block_dequant_gb300 import build

    build.build()
    qg.load()
    return qg


def cache(qg, **kw):
    c = dict(k=A, v=A, dtype=1, n_pages=8, page_size=16, n_heads=2, head_dim=128, page_stride=16 * 256,
             token_stride=256, head_stride=128)
    c.update(kw)
    return qg.KVCache(*[c[f] for f, _ in qg.KVCache._fields_])


def batch(qg, **kw):
    b = dict(n_seqs=3, n_tokens=3, n_groups=0, max_pages=4, max_prefix_pages=0, q_start=None, kv_len=A, pages=A,
             group_start=None, prefix_len=None, prefix_pages=None)
    b.update(kw)
    return qg.KVBatch(*[b[f] for f, _ in qg.KVBatch._fields_])


BAD_CACHES = [
    (dict(k=None), PTR), (dict(v=None), PTR), (dict(dtype=0), UNSUP), (dict(dtype=3), UNSUP),
    (dict(head_dim=96), UNSUP), (dict(head_dim=0), UNSUP), (dict(n_pages=0), SHAPE), (dict(page_size=0), SHAPE),
    (dict(page_size=24), SHAPE), (dict(page_size=1 << 17), SHAPE), (dict(n_heads=0), SHAPE),
    (dict(token_stride=-256), SHAPE), (dict(page_stride=1 << 50), SHAPE), (dict(k=ODD), ALIGN),
    (dict(head_stride=132), ALIGN), (dict(token_stride=258), ALIGN),
]
BAD_BATCHES = [
    (dict(kv_len=None), PTR), (dict(pages=None), PTR), (dict(n_seqs=-1), SHAPE), (dict(n_seqs=70000), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(n_tokens=4), SHAPE), (dict(n_tokens=-1, q_start=A), SHAPE),
    (dict(n_tokens=1 << 25, q_start=A), SHAPE), (dict(kv_len=ODD), ALIGN), (dict(q_start=ODD), ALIGN),
    (dict(n_groups=4, group_start=A, prefix_len=A, prefix_pages=A, max_prefix_pages=1), SHAPE),
    (dict(n_groups=1), PTR), (dict(n_groups=1, group_start=A, prefix_len=ODD, prefix_pages=A, max_prefix_pages=1), ALIGN),
]


def append(qg, c, b, Hq=4, q=A, qs=512, k=A, ks=256, v=A, vs=256, qn=None, kn=None, eps=1e-6, fr=A, rot=128, pairs=0,
           out=A):
    return qg.load().qg_kv_append(ctypes.byref(c), ctypes.byref(b), Hq, q, qs, k, ks, v, vs, qn, kn, eps, fr, rot, pairs,
                                  out, None)


def attend(qg, c, b, Hq=4, q=A, qs=512, scale=0.1, out=A, dt=0, ws=A, n=1 << 40):
    return qg.load().qg_attn_paged(ctypes.byref(c), ctypes.byref(b), Hq, q, qs, scale, out, dt, ws, n, None)


def test_caches_and_batches_are_checked(qg):
    for kw, want in BAD_CACHES:
        assert append(qg, cache(qg, **kw), batch(qg)) == want, kw
        assert attend(qg, cache(qg, **kw), batch(qg)) == want, kw
        assert qg.load().qg_beam_reorder(ctypes.byref(cache(qg, **kw)), 1, ctypes.byref(batch(qg)), 3, A, None) == want, kw
        assert qg.attn_workspace_size(cache(qg, **kw), batch(qg), 4) == 0
    for kw, want in BAD_BATCHES:
        assert append(qg, cache(qg), batch(qg, **kw)) == want, kw
        assert attend(qg, cache(qg), batch(qg, **kw)) == want, kw
    # the append does not read the prefix pages, attention does
    g = dict(n_groups=1, group_start=A, prefix_len=A)
    assert attend(qg, cache(qg), batch(qg, **g)) == PTR
    assert append(qg, cache(qg), batch(qg, n_seqs=0, n_tokens=0)) == 0  # nothing to do
    assert append(qg, cache(qg), batch(qg, **g, n_tokens=0, q_start=A)) == 0
    L = qg.load()
    assert L.qg_kv_append(None, ctypes.byref(batch(qg)), 4, A, 512, A, 256, A, 256, None, None, 0.0, A, 128, 0, A, None) == PTR
    assert L.qg_attn_paged(ctypes.byref(cache(qg)), None, 4, A, 512, 0.1, A, 0, A, 1 << 40, None) == PTR


def test_append_arguments(qg):
    c, b = cache(qg), batch(qg)
    for kw, want in [
        (dict(Hq=3), SHAPE), (dict(Hq=-2), SHAPE), (dict(rot=130), SHAPE), (dict(rot=136), SHAPE), (dict(rot=12), SHAPE),
        (dict(rot=-8), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=math.nan), SHAPE), (dict(pairs=2), SHAPE),
        (dict(q=None), PTR), (dict(out=None), PTR), (dict(k=None), PTR), (dict(v=None), PTR), (dict(fr=None), PTR),
        (dict(qs=508), SHAPE), (dict(ks=128), SHAPE), (dict(vs=0), SHAPE), (dict(qs=-512), SHAPE), (dict(qs=514), ALIGN),
        (dict(q=ODD), ALIGN), (dict(out=A + 8), ALIGN), (dict(fr=A + 4), ALIGN), (dict(qn=ODD), ALIGN), (dict(kn=A + 4), ALIGN),
    ]:
        assert append(qg, c, b, **kw) == want, kw


def test_attention_arguments(qg):
    c, b = cache(qg), batch(qg)
    need = qg.attn_workspace_size(c, b, 4)
    assert need > 0
    for kw, want in [
        (dict(Hq=3), SHAPE), (dict(Hq=0), SHAPE), (dict(Hq=34), UNSUP), (dict(q=None), PTR), (dict(out=None), PTR),
        (dict(dt=2), UNSUP), (dict(dt=7), UNSUP), (dict(scale=math.inf), SHAPE), (dict(scale=math.nan), SHAPE),
        (dict(qs=504), SHAPE), (dict(qs=516), ALIGN), (dict(q=ODD), ALIGN), (dict(out=A + 4), ALIGN), (dict(ws=None), WS),
        (dict(n=need - 1), WS), (dict(ws=A + 8), ALIGN),
    ]:
        assert attend(qg, c, b, **kw) == want, kw
    assert attend(qg, c, batch(qg, n_seqs=0, n_tokens=0)) == 0
    # a larger batch never needs less
    sizes = [qg.attn_workspace_size(c, batch(qg, n_seqs=n, n_tokens=t, q_start=A), 4)
             for n, t in ((1, 1), (1, 100), (4, 100), (4, 5000), (64, 5000))]
    assert sizes == sorted(sizes)


def test_select_arguments(qg):
    L = qg.load()

    def sel(x=A, s=A, d=None, eos=-1, N=2, W=3, K=4, V=100, o=A, p=A, t=A, ws=A, n=1 << 40):
        return L.qg_beam_select(x, s, d, eos, N, W, K, V, o, p, t, None, ws, n, None)

    for kw, want in [
        (dict(W=0), SHAPE), (dict(W=65), SHAPE), (dict(K=0), SHAPE), (dict(K=65), SHAPE), (dict(V=0), SHAPE),
        (dict(V=(1 << 20) + 1), SHAPE), (dict(K=4, W=3, V=1), SHAPE), (dict(N=-1), SHAPE), (dict(N=40000), SHAPE),
        (dict(eos=100), SHAPE), (dict(x=None), PTR), (dict(s=None), PTR), (dict(o=None), PTR), (dict(p=None), PTR),
        (dict(t=None), PTR), (dict(x=ODD), ALIGN), (dict(t=ODD), ALIGN), (dict(ws=None), WS), (dict(n=8), WS),
        (dict(ws=A + 4), ALIGN), (dict(N=0), 0),
    ]:
        assert sel(**kw) == want, kw
    assert qg.beam_workspace_size(2, 0, 4, 100) == 0
    assert qg.beam_workspace_size(2, 3, 4, 100) < qg.beam_workspace_size(2, 3, 4, 151936)


def test_reorder_arguments(qg):
    L = qg.load()
    cs = (qg.KVCache * 2)(cache(qg), cache(qg))

    def reo(c=cs, n=2, b=None, W=3, p=A):
        return L.qg_beam_reorder(c, n, ctypes.byref(b or batch(qg)), W, p, None)

    for kw, want in [(dict(n=0), SHAPE), (dict(n=129), SHAPE), (dict(W=0), SHAPE), (dict(W=33), SHAPE), (dict(W=2), SHAPE),
                     (dict(p=None), PTR), (dict(c=None), PTR), (dict(p=ODD), ALIGN), (dict(W=1), 0),
                     (dict(b=batch(qg, n_seqs=0)), 0), (dict(b=batch(qg, kv_len=None)), PTR)]:
        assert reo(**kw) == want, kw
    for kw in (dict(head_dim=64), dict(n_pages=9), dict(dtype=2), dict(token_stride=512)):
        assert reo(c=(qg.KVCache * 2)(cache(qg), cache(qg, **kw))) == SHAPE, kw


def test_rotation_table(qg):
    """Entry i is theta^(-2i/rot) / (2 pi) turns in units of 2^-64: half a unit, and the roundings of
    the double it is formed in."""
    for rot, theta in ((128, 1e6), (64, 10000.0), (2, 1.5)):
        t = qg.rope_freqs(rot, theta).tolist()
        for i, x in enumerate(t):
            want = theta ** (-2.0 * i / rot) / (2 * math.pi)
            assert abs((x % (1 << 64)) / 2.0 ** 64 - want) <= want * 2.0 ** -50 + 2.0 ** -65
    L, out = qg.load(), (ctypes.c_uint64 * 64)()
    fac = (F * 4)(1, 1, 0.1, 1)
    assert L.qg_rope_freqs(0, 1e4, None, out) == SHAPE and L.qg_rope_freqs(7, 1e4, None, out) == SHAPE
    assert L.qg_rope_freqs(8, 1.0, None, out) == SHAPE and L.qg_rope_freqs(8, math.inf, None, out) == SHAPE
    assert L.qg_rope_freqs(8, 1e4, None, None) == PTR
    assert L.qg_rope_freqs(8, 1e4, fac, out) == 0
    fac[0] = 0.0
    assert L.qg_rope_freqs(8, 1e4, fac, out) == SHAPE  # no such frequency
    fac[0] = 0.1
    assert L.qg_rope_freqs(8, 1e4, fac, out) == SHAPE  # more than a turn per position


def test_binding_checks(qg):
    torch = pytest.importorskip("torch")
    k = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    c = qg.kv_cache(k, k.clone())
    assert (c.n_pages, c.page_size, c.n_heads, c.head_dim) == (4, 16, 2, 64)
    h = torch.zeros((4, 2, 16, 64), dtype=torch.float16).permute(0, 2, 1, 3)
    c = qg.kv_cache(h, h.clone(memory_format=torch.preserve_format))
    assert (c.token_stride, c.head_stride, c.page_size) == (64, 1024, 16)
    for a, b in ((k, k[:2]), (k, k.bfloat16()), (k, h), (k[..., ::2], k[..., ::2]), (k[0], k[0]), (k.double(), k.double())):
        with pytest.raises(ValueError):
            qg.kv_cache(a, b)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    b = qg.kv_batch(i32(3), i32(3, 5), i32(4), 7, i32(2), i32(1), i32(1, 2))
    assert (b.n_seqs, b.n_tokens, b.n_groups, b.max_pages, b.max_prefix_pages) == (3, 7, 1, 5, 2)
    for args in ((i32(3), i32(2, 5)), (i32(3).long(), i32(3, 5)), (i32(3), i32(3, 10)[:, ::2]), (i32(3), i32(3, 5), i32(3), 7),
                 (i32(3), i32(3, 5), i32(4), None), (i32(3), i32(3, 5), None, 4), (i32(3), i32(3, 5), None, 3, None, i32(1)),
                 (i32(3), i32(3, 5), None, 3, i32(2), i32(1), i32(2, 2))):
        with pytest.raises(ValueError):
            qg.kv_batch(*args)


def test_binding_refuses_tensors_of_other_types_and_shapes(qg):
    """What the C side cannot see: a tensor of another type would be read past its end."""
    torch = pytest.importorskip("torch")
    k = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    c = qg.kv_cache(k, k.clone())
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    b = qg.kv_batch(i32(3), i32(3, 5))
    q, kv, qo, fr = torch.zeros(3, 256), torch.zeros(3, 128), torch.zeros((3, 4, 64), dtype=torch.float16), qg.rope_freqs(64, 1e4)
    bad = [dict(q=q.double()), dict(q=q[:2]), dict(q=torch.zeros(3, 192)), dict(k=kv.half()), dict(v=kv[:, :64]),
           dict(k=torch.zeros(128, 3).T), dict(q_out=qo.float()), dict(q_out=qo.transpose(0, 1)), dict(freqs=fr.float()),
           dict(q_norm=torch.zeros(32)), dict(k_norm=torch.zeros(64, dtype=torch.float64)),
           dict(q_out=torch.zeros(800, dtype=torch.float16))]
    for kw in bad:
        a = dict(q=q, k=kv, v=kv, q_out=qo, freqs=fr)
        a.update(kw)
        with pytest.raises(ValueError):
            qg.kv_append(c, b, stream=0, **a)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for qq, oo in ((qo.float(), qo), (qo[:2], qo), (qo, torch.zeros(3, 300)), (qo, torch.zeros(4, 64, 3).permute(2, 0, 1)),
                   (qo, qo.double())):
        with pytest.raises(ValueError):
            qg.attn_paged(c, b, qq, oo, 0.1, ws, stream=0)
    f, i, u = (torch.zeros(2, 3, dtype=t) for t in (torch.float32, torch.int32, torch.uint8))
    x = torch.zeros(6, 50)
    for kw in (dict(logits=x.half()), dict(logits=x[:5]), dict(logits=torch.zeros(50, 6).T), dict(scores=f.double()),
               dict(scores=f[0]), dict(out_scores=f.half()), dict(parents=i.long()), dict(tokens=f), dict(tokens=i[0]),
               dict(done=i), dict(done=u[0]), dict(done_out=i)):
        a = dict(logits=x, scores=f, N=2, W=3, out_scores=f, parents=i, tokens=i, workspace=ws, stream=0)
        a.update(kw)
        with pytest.raises(ValueError):
            qg.beam_select(**a)
    for p in (i32(2), i32(3).long(), torch.zeros(3)):
        with pytest.raises(ValueError):
            qg.beam_reorder(qg.kv_caches([k], [k.clone()]), b, p, 3, stream=0)


def test_binding_refuses_tensors_off_the_gpu(qg):
    """Host tensors (rope_freqs returns one) and those of another GPU are refused before the C call,
    which sees addresses only.  A subclass stands in for tensors of a GPU; nothing is called with it."""
    torch = pytest.importorskip("torch")

    class There(torch.Tensor):
        where = 0

        def get_device(self):
            return self.where

    class Elsewhere(There):
        where = 1

    g = lambda t: t.as_subclass(There)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    c, caches = qg.kv_cache(g(k), g(k.clone())), qg.kv_caches([g(k)], [g(k.clone())])
    b = qg.kv_batch(g(i32(3)), g(i32(3, 5)))
    assert c.device == b.device == caches.device == caches[0].device == [x.device for x in caches][0] == 0
    host = qg.kv_cache(k, k.clone())
    hostb = qg.kv_batch(i32(3), i32(3, 5))
    away = qg.kv_batch(i32(3).as_subclass(Elsewhere), i32(3, 5))
    f32 = lambda *s: g(torch.zeros(s))  # noqa: E731
    qo, ws = g(torch.zeros((3, 4, 64), dtype=torch.float16)), g(torch.zeros(1 << 20, dtype=torch.uint8))
    plain = lambda t: t.as_subclass(torch.Tensor)  # noqa: E731

    def refused(f, args, names, what):
        for n in names:
            for to in (plain, lambda t: t.as_subclass(Elsewhere)):
                a = dict(args)
                a[n] = to(a[n])
                with pytest.raises(ValueError, match=f"{what.get(n, n)} must be on"):
                    f(**a)

    a = dict(cache=c, batch=b, q=f32(3, 256), k=f32(3, 128), v=f32(3, 128), q_out=qo, freqs=g(qg.rope_freqs(64, 1e4)),
             q_norm=f32(64), k_norm=f32(64), stream=0)
    refused(qg.kv_append, a, ["q", "k", "v", "q_out", "freqs", "q_norm", "k_norm"], {})
    for kw in (dict(cache=host, batch=hostb), dict(batch=hostb), dict(batch=away)):
        with pytest.raises(ValueError, match="GPU"):
            qg.kv_append(**{**a, **kw})
    a = dict(cache=c, batch=b, q=qo, out=g(torch.zeros((3, 4, 64))), scale=0.1, workspace=ws, stream=0)
    refused(qg.attn_paged, a, ["q", "out", "workspace"], {})
    for kw in (dict(cache=host, batch=hostb), dict(batch=hostb), dict(cache=host)):
        with pytest.raises(ValueError, match="GPU"):
            qg.attn_paged(**{**a, **kw})
    gi, gu = g(i32(2, 3)), g(torch.zeros((2, 3), dtype=torch.uint8))
    a = dict(logits=f32(6, 50), scores=f32(2, 3), N=2, W=3, out_scores=f32(2, 3), parents=gi, tokens=gi, workspace=ws,
             done=gu, done_out=gu, stream=0)
    refused(qg.beam_select, a, ["scores", "out_scores", "parents", "tokens", "workspace", "done", "done_out"], {})
    with pytest.raises(ValueError, match="GPU"):
        qg.beam_select(**{**a, "logits": plain(a["logits"])})
    refused(lambda **kw: qg.beam_reorder(caches, b, W=3, stream=0, **kw), dict(parents=g(i32(3))), ["parents"], {})
    for cs, bb in ((caches, hostb), (qg.kv_caches([k], [k.clone()]), b)):
        with pytest.raises(ValueError, match="GPU"):
            qg.beam_reorder(cs, bb, g(i32(3)), 3, stream=0)
    with pytest.raises(ValueError, match="one device"):
        qg.kv_caches([g(k), k], [g(k), k])
    # what was refused for its type or shape still is, with every tensor in place
    good = dict(cache=c, batch=b, q=f32(3, 256), k=f32(3, 128), v=f32(3, 128), q_out=qo, freqs=g(qg.rope_freqs(64, 1e4)), stream=0)
    for kw, msg in ((dict(q=f32(3, 256).double()), "f32"), (dict(k=f32(3, 64)), "k must have"),
                    (dict(q_out=g(torch.zeros(3, 4, 64))), "cache's type"), (dict(q_norm=f32(32)), "head_dim")):
        with pytest.raises(ValueError, match=msg):
            qg.kv_append(**{**good, **kw})


def test_workspace_counts_a_prompts_tiles_once(qg):
    """A long prompt's tokens are in its own row tiles and in no run of a group: a shared prefix before it
    adds what the group's runs may need, not the prompt's tiles again."""
    c = cache(qg, n_heads=8, head_stride=128, token_stride=1024, page_stride=16 * 1024)
    g = dict(n_groups=1, group_start=A, prefix_len=A, prefix_pages=A, max_prefix_pages=4)
    for n, T in ((1, 131072), (4, 20000), (64, 5000)):
        one = qg.attn_workspace_size(c, batch(qg, n_seqs=n, n_tokens=T, q_start=A), 32)
        both = qg.attn_workspace_size(c, batch(qg, n_seqs=n, n_tokens=T, q_start=A, **g), 32)
        # a run per group and one after each long sequence, each a row tile of 256 rows and one of 16, per cached head
        assert one < both <= one + (n + 1) * 8 * (256 + 16) * (128 + 2) * 4 + (1 << 16)
