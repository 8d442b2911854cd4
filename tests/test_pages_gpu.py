"""Pages with holders on the GPU: fork, reserve and compact against plain lists."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


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


class Server:
    """Caches of some layers, page lists and counts, here as lists and on the GPU as the library sees them."""

    def __init__(self, qg, n_pages, B, cols, page=16, layers=2, Hkv=2, D=64, dtype="f16", layout="nhd", seed=0):
        self.qg, self.page, self.cols, self.n_pages, self.B = qg, page, cols, n_pages, B
        g = torch.Generator().manual_seed(seed)
        dims = (page, Hkv) if layout == "nhd" else (Hkv, page)
        self.pool = torch.randn((2 * layers, n_pages, *dims, D), generator=g).to(DT[dtype])
        d = self.pool.cuda()
        self.view = (lambda p: p) if layout == "nhd" else (lambda p: p.permute(0, 1, 3, 2, 4))
        self.dpool = d
        v = self.view(d)
        self.caches = qg.kv_caches(list(v[0::2]), list(v[1::2]))
        self.kv, self.refs = [0] * B, [0] * n_pages
        self.table = [[-9] * cols for _ in range(B)]  # what nobody holds stays as it is

    def up(self):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.dkv, self.drefs, self.dtable = i32(self.kv), i32(self.refs), i32(self.table)
        self.batch = self.qg.kv_batch(self.dkv, self.dtable.reshape(self.B, self.cols))
        self.missing = torch.full((1,), -5, dtype=torch.int32, device="cuda")
        self.ws = torch.full((self.qg.reserve_workspace_size(self.caches, self.batch),), 255, dtype=torch.uint8, device="cuda")
        return self

    def held(self, b):
        return -(-self.kv[b] // self.page)

    # -- the definitions
    def fork(self, src=None, keep=None):
        src = list(range(self.B)) if src is None else src
        old_kv = list(self.kv)
        for b, s in enumerate(src):
            k = -1 if keep is None else keep[b]
            length = 0 if s < 0 else old_kv[s]
            length = length if k < 0 else min(k, length)
            n = -(-length // self.page)
            for i in range(n if s == b else 0, -(-old_kv[b] // self.page)):
                self.refs[self.table[b][i]] -= 1
            if s >= 0 and s != b:
                for i in range(n):
                    self.table[b][i] = self.table[s][i]
                    self.refs[self.table[s][i]] += 1
            self.kv[b] = length

    def reserve(self, add):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        many = [r > 1 for r in self.refs]
        plan = []
        for b in range(self.B):
            full, rem = divmod(self.kv[b], self.page)
            copy = bool(add[b] and rem and many[self.table[b][full]])
            cols = ([full] if copy else []) + list(range(self.held(b), -(-(self.kv[b] + add[b]) // self.page)) if add[b] else [])
            plan.append((b, copy, full, rem, cols))
        need = sum(len(p[4]) for p in plan)
        if need > len(free):
            return need - len(free)
        view, at = self.view(self.pool), 0
        for b, copy, full, rem, cols in plan:
            old = self.table[b][full] if copy else None
            for c in cols:
                self.table[b][c] = free[at]
                self.refs[free[at]] = 1
                at += 1
            if copy:
                self.refs[old] -= 1
                view[:, self.table[b][full], :rem] = view[:, old, :rem]
            self.kv[b] += add[b]
        return 0

    def compact(self, src, start, keep):
        view = self.view(self.pool)
        for b, s in enumerate(src):
            if s >= 0:
                for i, slot in enumerate(keep[start[b]:start[b + 1]]):
                    view[:, self.table[b][i // self.page], i % self.page] = view[:, self.table[s][slot // self.page], slot % self.page]

    def call(self, name, *args, **kw):
        i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        if name == "fork":
            self.qg.kv_fork(self.caches, self.batch, self.drefs, src=i32(kw.get("src")), keep=i32(kw.get("keep")))
        elif name == "reserve":
            self.qg.kv_reserve(self.caches, self.batch, self.drefs, i32(args[0]), self.missing, self.ws)
        else:
            self.qg.kv_compact(self.caches, self.batch, *[i32(a) for a in args])

    def same(self, status=0):
        assert self.dkv.tolist() == self.kv
        assert self.drefs.tolist() == self.refs
        assert self.dtable.tolist() == self.table
        assert torch.equal(self.dpool.cpu().view(torch.int16), self.pool.view(torch.int16))
        assert self.qg.device_status() == status


CACHES = [dict(), dict(page=1, D=128, dtype="bf16"), dict(page=8, Hkv=1, layout="hnd"), dict(page=64, layers=5, Hkv=4, D=256, layout="hnd"),
          dict(page=32, layers=1, Hkv=3, D=128)]


@pytest.mark.parametrize("kw", CACHES, ids=str)
def test_a_server_run(qg, kw):
    """Prompts, forks of them, drafts that come and go, sequences that end: many random rounds."""
    r = random.Random(len(str(kw)))
    s = Server(qg, n_pages=60, B=9, cols=40, **kw).up()
    missed = 0
    for step in range(60):
        what = r.random()
        src, keep = list(range(9)), [-1] * 9
        if what < 0.35:
            sources = r.sample(range(9), 4)
            for b in range(9):
                if b not in sources and r.random() < 0.4:
                    src[b] = r.choice([-1, *sources])
                    keep[b] = r.choice([-1, -1, r.randint(0, 40), 10 ** 6])
            s.fork(src, keep)
            s.call("fork", src=src, keep=keep)
        elif what < 0.6:
            keep = [r.choice([-1, max(0, x - r.randint(0, 5)), x + 3, 0 if r.random() < 0.2 else x]) for x in s.kv]
            s.fork(None, keep)
            s.call("fork", keep=keep)
        else:
            room = [s.cols * s.page - x for x in s.kv]
            add = [min(room[b], r.choice([0, 1, 1, 2, 5, r.randint(0, 3 * s.page)])) for b in range(9)]
            short = s.reserve(add)
            s.call("reserve", add)
            assert s.missing.item() == short
            missed += short > 0
        s.same()
    assert missed < 40


def test_reserve_too_few_pages_changes_nothing(qg):
    s = Server(qg, n_pages=6, B=3, cols=8)
    s.kv, s.refs = [20, 20, 0], [0, 2, 2, 0, 0, 0]
    s.table[0][:2] = s.table[1][:2] = [1, 2]
    s.up()
    s.call("reserve", [1, 1, 40])
    assert s.missing.item() == 1  # two copies and three pages, four are free
    s.same()
    assert s.reserve([1, 1, 30]) == 0
    s.call("reserve", [1, 1, 30])
    assert s.missing.item() == 0
    s.same()
    assert s.refs[2] == 0  # both holders have their own now


@pytest.mark.parametrize("side", [False, True])
def test_reserve_without_sequences(qg, side):
    """Nothing is missing where nothing is asked for: a server whose last sequence has just left."""
    s = Server(qg, n_pages=6, B=0, cols=8)
    s.refs = [0, 2, 1, 0, 0, 0]
    s.up()
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    qg.kv_reserve(s.caches, s.batch, s.drefs, none, s.missing, s.ws, stream=stream)
    torch.cuda.synchronize()
    assert s.missing.item() == 0 and s.drefs.tolist() == s.refs


def test_every_holder_copies(qg):
    """Sixteen continuations of one prompt, the prompt going on as well."""
    s = Server(qg, n_pages=300, B=17, cols=8, layers=3, D=128, seed=1)
    s.reserve([45] + [0] * 16)
    s.up()
    s.fork([0] * 17, None)
    s.call("fork", src=[0] * 17)
    s.same()
    add = [1 + b % 4 for b in range(17)]
    assert s.reserve(add) == 0
    s.call("reserve", add)
    s.same()


def test_many_sequences_and_pages(qg):
    """More sequences and pages than one block's threads, free pages far behind."""
    B, cols = 3000, 4
    r = random.Random(5)
    s = Server(qg, n_pages=13000, B=B, cols=cols, page=2, layers=1, Hkv=1, seed=2)
    s.reserve([r.randint(0, 5) for _ in range(B)])
    src, keep = list(range(B)), [-1] * B
    for b in range(1000, 2000):
        src[b] = r.choice([-1, b - 1000])
    s.fork(src, keep)
    s.up()
    add = [r.randint(0, 2) for _ in range(B)]
    assert s.reserve(add) == 0
    s.call("reserve", add)
    s.same()
    s.fork([-1] * B, None)
    s.call("fork", src=[-1] * B)
    s.same()
    assert not any(s.refs)


@pytest.mark.parametrize("bad", ["source changes", "source truncated", "source outside", "keep", "long", "negative length", "page", "count"])
def test_fork_refuses(qg, bad):
    """What cannot be done leaves its sequence as it is; the others are done."""
    s = Server(qg, n_pages=20, B=5, cols=4)
    s.reserve([30, 20, 17, 5, 0])
    src, keep = [0, 1, 0, 3, 1], [-1, -1, -1, 2, -1]
    ok = list(src)
    okk = list(keep)
    status = 1 << qg.QG_EDEVICE_ID
    if bad == "source changes":
        src[1], src[4] = 0, 1
        ok[1], ok[4] = 0, 4
    elif bad == "source truncated":
        keep[1] = 3
        ok[4], okk[1] = 4, 3
    elif bad == "source outside":
        src[2], src[4], ok[2], ok[4] = 5, -2, 2, 4
    elif bad == "keep":
        keep[2], ok[2], okk[2] = -2, 2, -1
    elif bad in ("long", "negative length"):
        s.kv[4] = 65 if bad == "long" else -3
        ok[4] = 4
    elif bad == "page":
        s.table[3][0] = 99
    elif bad == "count":
        s.refs[s.table[2][1]] = 0
    s.up()
    kv4 = s.kv[4]
    if ok[4] == 4:
        s.kv[4] = 0
    if bad == "page":
        s.up()
        keep[3] = okk[3] = 0
        hold = list(s.refs)
        s.table[3][0] = 0
        s.fork(ok, okk)
        s.refs[0] += 1  # the page outside is not counted: 0's release was not one
        s.table[3][0] = 99
        assert hold
    elif bad == "count":
        s.refs[s.table[2][1]] = 1
        s.fork(ok, okk)
    else:
        s.fork(ok, okk)
    if ok[4] == 4:
        s.kv[4] = kv4
    s.call("fork", src=src, keep=keep)
    s.same(status)


@pytest.mark.parametrize("bad", ["add", "list", "length", "page"])
def test_reserve_refuses(qg, bad):
    s = Server(qg, n_pages=20, B=3, cols=3)
    s.reserve([20, 20, 20])
    add, ok = [7, 7, 20], [7, 7, 20]
    ok[1] = 0
    if bad == "add":
        add[1] = -1
    elif bad == "list":
        add[1] = 29
    elif bad == "length":
        s.kv[1] = -4
    else:
        s.table[1][1] = 20
    s.up()
    hold = s.kv[1], list(s.table[1])
    s.kv[1] = 0
    assert s.reserve(ok) == 0
    s.kv[1], s.table[1] = hold
    s.call("reserve", add)
    assert s.missing.item() == 0
    s.same(1 << qg.QG_EDEVICE_ID)


@pytest.mark.parametrize("kw", CACHES, ids=str)
def test_compact(qg, kw):
    """Some tokens of some sequences, none of others, one context to several receivers."""
    r = random.Random(9)
    s = Server(qg, n_pages=400, B=7, cols=90, seed=3, **kw)
    s.reserve([90, 33, 1, 60, 20, 0, 5])
    s.up()
    src = [-1, -1, -1, 0, 1, -1, 0]
    lists = [[], [], [], sorted(r.sample(range(90), 60)), [32], [], [7, 3, 3, 89]]  # any order, one token twice
    start = [0]
    for x in lists:
        start.append(start[-1] + len(x))
    keep = [i for x in lists for i in x]
    s.compact(src, start, keep)
    s.call("compact", src, start, keep)
    s.same()


def test_compact_refuses(qg):
    """Tokens that are not there, receivers without room, a sequence to itself, pages outside the pool."""
    s = Server(qg, n_pages=40, B=6, cols=4, seed=4)
    s.reserve([40, 20, 2, 20, 20, 20])
    s.up()
    cases = [([-1, 0, -1, -1, -1, -1], [0, 0, 4, 4, 4, 4, 4], [1, 40, -1, 39], [0, 3]),
             ([-1, -1, 0, -1, -1, -1], [0, 0, 0, 4, 4, 4, 4], [5, 6, 7, 8], [0, 1]),
             ([0, 6, -2, -1, -1, -1], [0, 2, 4, 6, 6, 6, 6], [1, 2, 3, 4, 5, 6], [])]
    for src, start, keep, good in cases:
        b = next((i for i, x in enumerate(src) if x == 0 and i), None)
        for i in good:
            s.view(s.pool)[:, s.table[b][i // 16], i % 16] = s.view(s.pool)[:, s.table[0][keep[i] // 16], keep[i] % 16]
        s.call("compact", src, start, keep)
        s.same(1 << qg.QG_EDEVICE_ID)
    s.table[3][0], s.table[0][1] = 40, -1
    s.up()
    s.call("compact", [-1, -1, -1, 0, 0, -1], [0, 0, 0, 0, 2, 5, 5], [3, 4, 2, 17, 3])
    for i, k in ((0, 2), (2, 3)):
        s.view(s.pool)[:, s.table[4][0], i] = s.view(s.pool)[:, s.table[0][0], k]
    s.same(1 << qg.QG_EDEVICE_ID)
    s.call("compact", [-1, -1, -1, -1, -1, 4], [0, -7, 90, 3, 5, 0, 1 << 20], [3, 4])  # starts that do not rise: nothing outside
    qg.device_status()


def test_far_pages(qg):
    """Pages whose offsets pass 32 bits."""
    n_pages, page, Hkv, D = 20000, 128, 8, 128  # 2^17 elements a page, 5 GB a pool
    pool = torch.zeros((2, n_pages, page, Hkv, D), dtype=torch.float16, device="cuda")
    pool[:, n_pages - 3, :9] = torch.randn((2, 9, Hkv, D), device="cuda").half()
    caches = qg.kv_caches([pool[0]], [pool[1]])
    refs = torch.ones((n_pages,), dtype=torch.int32, device="cuda")
    refs[n_pages - 3] = 2
    refs[n_pages - 2:] = 0
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kv, table = i32([9, 9]), i32([[n_pages - 3], [n_pages - 3]])
    batch = qg.kv_batch(kv, table)
    ws = torch.empty(qg.reserve_workspace_size(caches, batch), dtype=torch.uint8, device="cuda")
    missing = i32([0])
    qg.kv_reserve(caches, batch, refs, i32([2, 0]), missing, ws)
    assert table.tolist() == [[n_pages - 2], [n_pages - 3]] and refs[-3:].tolist() == [1, 1, 0] and kv.tolist() == [11, 9]
    assert torch.equal(pool[:, n_pages - 2, :9], pool[:, n_pages - 3, :9]) and not pool[:, n_pages - 2, 9:].any()
    qg.kv_compact(caches, batch, i32([1, -1]), i32([0, 2, 2]), i32([8, 4]))
    assert torch.equal(pool[:, n_pages - 2, :2], pool[:, n_pages - 3, [8, 4]])
    assert qg.device_status() == 0


def test_graph_and_stream(qg):
    """Fork, reserve and compact captured in one graph on a side stream, replayed; a workspace full of old numbers."""
    s = Server(qg, n_pages=80, B=4, cols=6, layers=3, seed=6)
    s.reserve([37, 0, 0, 40])
    s.up()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    src, add = i32([0, 0, 0, 3]), i32([0, 3, 20, 0])
    csrc, start, keep = i32([-1, -1, -1, 1]), i32([0, 0, 0, 0, 3]), i32([39, 0, 20])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qg.kv_fork(s.caches, s.batch, s.drefs, src=src)
        qg.kv_reserve(s.caches, s.batch, s.drefs, add, s.missing, s.ws)
        qg.kv_compact(s.caches, s.batch, csrc, start, keep)
    for _ in range(3):
        s.fork([0, 0, 0, 3], None)
        assert s.reserve([0, 3, 20, 0]) == 0
        s.compact([-1, -1, -1, 1], [0, 0, 0, 0, 3], [39, 0, 20])
        graph.replay()
        torch.cuda.synchronize()
        s.same()


def test_more_pages_than_the_pool_has(qg):
    """What is missing is told in full where one sequence alone needs more pages than there are, and where many do."""
    s = Server(qg, n_pages=4, B=3, cols=5000, page=1, layers=1)
    s.up()
    for add in ([10, 0, 0], [5, 0, 0], [0, 4000, 4999], [3, 3, 0]):
        want = sum(add) - 4
        s.call("reserve", add)
        assert s.missing.item() == want
        s.same()
    s = Server(qg, n_pages=7, B=1200, cols=100, page=2, layers=1, Hkv=1)
    s.refs = [1] * 7
    s.up()
    s.call("reserve", [199 + b % 2 for b in range(1200)])
    assert s.missing.item() == 1200 * 100
    s.same()


def test_reserve_without_sequences_refuses_what_is_refused_otherwise(qg):
    """Caches of two geometries."""
    s = Server(qg, n_pages=6, B=0, cols=8)
    s.up()
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    k, k2 = (torch.zeros((6, 16, h, 64), dtype=torch.float16, device="cuda") for h in (2, 4))
    with pytest.raises(qg.QGError):
        qg.kv_reserve(qg.kv_caches([k, k2], [k, k2]), s.batch, s.drefs, none, s.missing, s.ws)
    assert s.missing.item() == -5


@pytest.mark.parametrize("start", [[0, -7, 90, 3, 5, 0, 1 << 20], [5, 4, 3, 2, 1, 0, -1], [-(1 << 31), 0, 0, 0, 0, 0, 2 ** 31 - 1], [9] * 7],
                         ids=str)
def test_compact_with_starts_that_do_not_rise(qg, start):
    """Lists, lengths and every page but the receiver's stay as they are, whatever its tokens are."""
    s = Server(qg, n_pages=40, B=6, cols=4, seed=7)
    s.reserve([40, 20, 2, 20, 20, 20])
    s.up()
    s.call("compact", [-1, -1, -1, -1, -1, 4], start, [3, 4])
    assert qg.device_status() in (0, 1 << qg.QG_EDEVICE_ID)
    held = s.table[5][:2]
    others = [p for p in range(40) if p not in held]
    assert (s.dkv.tolist(), s.drefs.tolist(), s.dtable.tolist()) == (s.kv, s.refs, s.table)
    assert torch.equal(s.dpool.cpu()[:, others].view(torch.int16), s.pool[:, others].view(torch.int16))
    # what the receiver's pages hold: tokens of the source, or what they held
    got, old = s.dpool.cpu()[:, held].flatten(1, 2), s.pool[:, held].flatten(1, 2)
    source = s.pool[:, s.table[4][0]][:, [3, 4]]
    for i in range(got.shape[1]):
        assert any(torch.equal(got[:, i], x) for x in (old[:, i], source[:, 0], source[:, 1]))
