"""The gated delta rule on the GPU against its definition in 64 bits."""
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


LENGTHS = [[1], [1, 1, 1], [5], [0, 3, 0, 1], [31, 32, 33], [64, 1, 0, 47], [17, 100], [257]]


@pytest.mark.parametrize("n", LENGTHS, ids=str)
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 32), (64, 96), (128, 256), (128, 64), (64, 128)])
def test_lengths_and_widths(qg, n, Dk, Dv):
    B = len(n)
    c = Delta(n, Dk=Dk, Dv=Dv, ins=[3 * b + 1 if b % 3 != 2 else -1 for b in range(B)], outs=[3 * b + 2 for b in range(B)], seed=B + n[0])
    c.check(c.run(qg))
    assert qg.device_status() == 0


@pytest.mark.parametrize("Dv", [128, 32])
def test_many_sequences(qg, Dv):
    """More sequences than are put in order, and than a round of the search looks at; lengths on both sides of the border."""
    n = [(7 * b) % 67 for b in range(150)]
    c = Delta(n, Hk=1, Hv=2, Dk=64, Dv=Dv, ins=[b if b % 4 else -1 for b in range(150)], outs=[150 + b for b in range(150)], seed=4)
    c.check(c.run(qg))
    assert qg.device_status() == 0


@pytest.mark.parametrize("n", [[0], [0, 0, 0]], ids=str)
def test_nothing_to_do(qg, n):
    c = Delta(n, Dv=32, ins=[0] * len(n), outs=[1] * len(n), behind=4, seed=3)
    c.check(c.run(qg))


@pytest.mark.parametrize("n", [[19, 20, 21], [52, 63, 65]], ids=str)
def test_later_magnitudes(qg, n):
    """Values that grow by a million within a chunk: earlier tokens keep their own precision."""
    c = Delta(n, ins=[0, 1, 2], outs=[3, 4, 5], seed=2)
    v = c.parts(c.x, c.ba)[2]
    v *= torch.logspace(-3, 3, c.T)[:, None, None]
    c.check(c.run(qg))


@pytest.mark.parametrize("Hk,Hv,tiled", [(1, 1, False), (3, 3, True), (2, 8, False), (2, 8, True), (16, 32, False)])
@pytest.mark.parametrize("raw,l2", [(True, True), (False, False), (False, True)])
def test_heads_and_gates(qg, Hk, Hv, tiled, raw, l2):
    c = Delta([40, 3], Hk=Hk, Hv=Hv, Dv=64, raw=raw, l2=l2, tiled=tiled, ins=[0, -1], outs=[1, 2], seed=Hv)
    c.check(c.run(qg))


@pytest.mark.parametrize("n", [[1, 1], [70, 2]], ids=str)
def test_a_slot_is_read_and_written(qg, n):
    c = Delta(n, ins=[2, 0], outs=[2, 0], behind=3, seed=5)
    c.check(c.run(qg))


def test_no_states(qg):
    c = Delta([4, 50], ins=None, outs=None, seed=6)
    c.check(c.run(qg))
    c = Delta([4, 50], ins=[-1, 0], outs=[-1, -1], seed=7)
    c.check(c.run(qg))


@pytest.mark.parametrize("n", [[3, 0, 6], [18, 40]], ids=str)
def test_states_kept_after_tokens(qg, n):
    """Each token's state, some of them not kept; a call from a kept state goes on as the whole run did."""
    T = sum(n)
    each = [i + 4 if i % 4 != 1 else -1 for i in range(T)]
    c = Delta(n, Dv=64, ins=[0, 1, -1][:len(n)], outs=[2, -1, 3][:len(n)], each=each, slots=T + 6, seed=8)
    c.check(c.run(qg))


@pytest.mark.parametrize("hint", [0, 1, 40, 1000])
def test_the_hint_changes_nothing(qg, hint):
    """max_new below, at and above what the sequences have."""
    c = Delta([40, 1, 33, 0], Dv=64, ins=[0, 1, 2, 3], outs=[4, 5, 6, 7], seed=9)
    c.check(c.run(qg, max_new=hint))


@pytest.mark.parametrize("n", [[6], [90]], ids=str)
def test_decay_extremes(qg, n):
    """No decay at all, decays that leave nothing (-inf among them), steps of 0, 1 and 2."""
    c = Delta(n, Dv=32, raw=False, l2=True, ins=[0], outs=[1], seed=10)
    T, Hv = n[0], c.Hv
    kinds = torch.tensor([0.0, -float("inf"), -1e30, -104.0, -12.0, -1e-6])
    g = torch.Generator().manual_seed(1)
    c.ba[:, :Hv] = kinds[torch.randint(0, len(kinds), (T, Hv), generator=g)]
    c.ba[:, 0] = 0.0
    c.ba[:, 1] = -11.0  # each token all but forgets the last, fifty chunks' worth of decay in one
    c.ba[:, Hv:2 * Hv] = torch.tensor([0.0, 1.0, 0.5, 2.0])[torch.randint(0, 4, (T, Hv), generator=g)]
    c.check(c.run(qg))


@pytest.mark.parametrize("big", [1e-30, 1e25])
def test_magnitudes(qg, big):
    """States and values far from 1, columns of very different size side by side."""
    c = Delta([50, 2], Dv=64, ins=[0, 1], outs=[2, 3], seed=11)
    f = torch.where(torch.arange(64) % 2 == 0, big, 1.0)
    c.states *= f
    v = c.parts(c.x, c.ba)[2]
    v *= f
    c.check(c.run(qg))


def test_zero_rows(qg):
    """Queries and keys of zeros: with the eps they stay zeros."""
    c = Delta([40, 1], Dv=32, ins=[0, 1], outs=[2, 3], seed=12)
    q, k, v, _, _ = c.parts(c.x, c.ba)
    q[3], k[7], k[40], v[9] = 0, 0, 0, 0
    c.check(c.run(qg))


@pytest.mark.parametrize("what", ["q", "k", "v", "a", "b"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [2, 45])
def test_nonfinite_tokens_reach_no_earlier_ones(qg, what, value, at):
    n = [70, 6, 40]
    c = Delta(n, Dv=64, ins=[0, 1, 2], outs=[3, 4, 5], raw=False, seed=13)
    clean = c.reference()
    h, j = 1, 33
    t = c.parts(c.x, c.ba)["qkvab".index(what)]
    if what in "qk":
        t[at, 0, 5] = value  # key head 0: value heads 0 and 1
        heads = [0, 1]
    elif what == "v":
        t[at, h, j] = value
        heads = [h]
    else:
        t[at, h] = value
        heads = [h]
    o, s = c.run(qg)
    o, s = o.double().cpu(), s.double().cpu()
    out, states, size, sizes = clean
    ok = (o - out).abs() <= 48 * 2.0 ** -24 * size * c.scale + 1e-37
    hit = torch.zeros_like(ok)
    cols = slice(j, j + 1) if what == "v" else slice(None)
    last = at + 1 if what == "q" else n[0]
    for x in heads:
        hit[at:last, x, cols] = True
    assert ok[~hit].all()
    if not (what == "a" and value > 0):  # a decay of +inf leaves zeros where the state is zero
        assert not torch.isfinite(o[hit]).any()
    sok = (s - states).abs() <= 48 * 2.0 ** -24 * sizes + 1e-37
    shit = torch.zeros_like(sok)
    if what != "q":
        for x in heads:
            shit[3, x, :, cols] = True
    assert sok[~shit].all()


def test_nonfinite_state_stays_in_its_columns(qg):
    c = Delta([40, 2], Dv=64, ins=[0, 1], outs=[2, 3], seed=14)
    want = c.reference()
    c.states[0, 1, 3, 7] = float("inf")
    c.states[1, 0, 9, 40] = float("nan")
    o = c.run(qg)[0].double().cpu()
    out, _, size, _ = want
    ok = (o - out).abs() <= 48 * 2.0 ** -24 * size * c.scale + 1e-37
    hit = torch.zeros_like(ok)
    hit[:40, 1, 7] = True
    hit[40:, 0, 40] = True
    assert ok[~hit].all() and not torch.isfinite(o[hit]).any()


def test_bad_slots(qg):
    """Slots outside the pool: the state in counts as none, the others are not kept, and the status says so."""
    c = Delta([3, 40, 2], Dv=32, ins=[0, 1, 2], outs=[3, 4, 5], slots=7, seed=15)
    ref = Delta([3, 40, 2], Dv=32, ins=[-1, 1, 2], outs=[3, -1, 5], slots=7, seed=15)
    c.ins, c.outs = [7, 1, 2], [3, 99, 5]
    got = c.run(qg)
    assert qg.device_status() == 1 << qg.QG_EDEVICE_ID
    ref.check(got)
    c.ins, c.outs = [-2, 1, 2], [3, -5, 5]
    ref.check(c.run(qg))
    assert qg.device_status() == 1 << qg.QG_EDEVICE_ID
    c = Delta([3], Dv=32, ins=[0], outs=[1], each=[2, 50, 3], slots=5, seed=16)
    got = c.run(qg)
    assert qg.device_status() == 1 << qg.QG_EDEVICE_ID
    c.each = [2, -1, 3]
    c.check(got)


def test_bad_starts_stay_inside(qg):
    """Starts that are negative, fall or pass the rows: rows and slots outside stay as they were."""
    c = Delta([20, 20, 20], Dv=32, ins=[0, 1, 2], outs=[3, 4, 5], seed=17)
    c.start = [-5, 70, 30, 1000]
    c.run(qg)
    torch.cuda.synchronize()


def test_far_slots(qg):
    """Slots whose offsets pass 32 bits."""
    Hv, D = 8, 128
    slots = 2 ** 31 // (Hv * D * D) + 40
    pool = torch.empty((slots, Hv, D, D), device="cuda")
    for n in ([1, 2], [70, 3]):
        c = Delta(n, Hk=4, Hv=Hv, ins=[0, 1], outs=[2, 3], seed=18)
        far = [slots - 1, slots - 4, slots - 2, 1]
        for i, s in enumerate(far):
            pool[s] = c.states[i].cuda()
        d = Delta(n, Hk=4, Hv=Hv, ins=[0, 1], outs=[2, 3], seed=18)
        d.ins, d.outs = far[:2], far[2:]
        out, _ = d.run(qg, states=pool)
        got = c.states.clone()
        for i, s in enumerate(far):
            got[i] = pool[s].cpu()
        c.check((out, got))


def test_chunks_and_tokens_agree(qg):
    """A prompt in one call, and in pieces that go through the other kernel."""
    whole = Delta([100], Dv=64, ins=[-1], outs=[0], slots=3, seed=19)
    o, s = whole.run(qg)
    states = whole.states.cuda()
    outs = []
    for i, (lo, hi) in enumerate([(0, 40), (40, 41), (41, 60), (60, 100)]):
        d = Delta([hi - lo], Dv=64, ins=[0 if lo else -1], outs=[0], slots=3, seed=19)
        d.x, d.ba = whole.x[lo:hi], whole.ba[lo:hi]
        d.a_scale, d.a_bias = whole.a_scale, whole.a_bias
        outs.append(d.run(qg, states=states)[0])
    whole.check((torch.cat(outs), states))
    whole.check((o, s))


@pytest.mark.parametrize("n", [[1] * 5, [3, 40, 70]], ids=str)
def test_streams_graphs_and_repetition(qg, n):
    """Another stream than the current one; a captured call replayed on new inputs; the same bits each time."""
    B = len(n)
    c = Delta(n, Dv=64, ins=list(range(B)), outs=list(range(B, 2 * B)), seed=20)
    first = [t.clone() for t in c.run(qg)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hold = []
    o, s = c.run(qg, stream=side, hold=hold)
    torch.cuda.synchronize()
    assert torch.equal(o, first[0]) and torch.equal(s, first[1])
    args, kw = hold
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg.delta_rule(*args, **kw)
    other = Delta(n, Dv=64, ins=c.ins, outs=c.outs, seed=21)
    q, k, v, a, b = other.parts(other.x.cuda(), other.ba.cuda())
    for dst, src in zip(args, (q, k, v, a, b, other.states.cuda())):
        dst.copy_(src)
    kw["a_scale"].copy_(other.a_scale)
    kw["a_bias"].copy_(other.a_bias)
    graph.replay()
    other.check((args[8], args[5]))


def test_two_streams_at_once(qg):
    a = Delta([300, 5], Dv=64, ins=[0, 1], outs=[2, 3], seed=22)
    b = Delta([200, 64], Dv=128, ins=[0, 1], outs=[2, 3], seed=23)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for c, s in ((a, s1), (b, s2)):
        with torch.cuda.stream(s):
            got.append(c.run(qg))
    torch.cuda.synchronize()
    a.check(got[0])
    b.check(got[1])
