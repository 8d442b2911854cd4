"""Paged caches, ragged batches and 64-bit references for the cached-decode tests."""
import math

import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


class Batch:
    """Page pools filled with random tokens, page lists over shuffled pages, and what a 64-bit
    reference needs.  `n`, `own`: new and cached tokens per sequence; `groups`: (first sequence,
    end, prefix length); rows no token owns hold `stale`."""

    def __init__(self, n, own, Hkv, D, page, dtype, groups=(), layout="nhd", stale=float("nan"), seed=0, spare=3,
                 extra_cols=1):
        g = torch.Generator().manual_seed(seed)
        self.n, self.own, self.groups, self.page, self.D, self.Hkv = list(n), list(own), list(groups), page, D, Hkv
        B = len(self.n)
        need = [-(-max(0, x) // page) for x in self.own] + [-(-max(0, x) // page) for _, _, x in self.groups]
        total = sum(need) + spare
        perm = torch.randperm(total, generator=g).tolist()
        dims = (page, Hkv, D) if layout == "nhd" else (Hkv, page, D)
        pools = [torch.full((total, *dims), stale, dtype=DT[dtype]) for _ in range(2)]
        if layout == "hnd":
            pools = [p.permute(0, 2, 1, 3) for p in pools]
        lists, at = [], 0
        for c in need:
            lists.append(perm[at:at + c])
            at += c
        self.rows = []  # (k, v) of each list in token order
        for ln, pages in zip([*self.own, *[x for _, _, x in self.groups]], lists):
            ln = max(0, ln)
            kv = [torch.randn((ln, Hkv, D), generator=g).to(DT[dtype]) for _ in range(2)]
            for s in range(ln):
                for p, x in zip(pools, kv):
                    p[pages[s // page], s % page] = x[s]
            self.rows.append(kv)
        # a permuted view keeps its strides on the device only if the base is moved
        if layout == "hnd":
            pools = [p.permute(0, 2, 1, 3).cuda().permute(0, 2, 1, 3) for p in pools]
        else:
            pools = [p.cuda() for p in pools]
        self.k, self.v = pools

        def table(ls, cols):
            t = torch.full((len(ls), max(1, cols)), -7, dtype=torch.int32)  # unused entries are no pages
            for i, x in enumerate(ls):
                t[i, :len(x)] = torch.tensor(x, dtype=torch.int32)
            return t.cuda()

        self.pages = table(lists[:B], max([len(x) for x in lists[:B]], default=0) + extra_cols)
        self.kv_len = torch.tensor(self.own, dtype=torch.int32).cuda()
        self.qs = [0]
        for x in self.n:
            self.qs.append(self.qs[-1] + x)
        self.T = self.qs[-1]
        self.q_start = torch.tensor(self.qs, dtype=torch.int32).cuda()
        self.group_start = self.prefix_len = self.prefix_pages = None
        if self.groups:
            self.group_start = torch.tensor([a for a, _, _ in self.groups] + [self.groups[-1][1]],
                                            dtype=torch.int32).cuda()
            self.prefix_len = torch.tensor([x for _, _, x in self.groups], dtype=torch.int32).cuda()
            self.prefix_pages = table(lists[B:], max(len(x) for x in lists[B:]))

    def desc(self, qg, plain_q=False):
        return qg.kv_batch(self.kv_len, self.pages, None if plain_q else self.q_start, self.T, self.group_start,
                           self.prefix_len, self.prefix_pages)

    def group(self, b):
        for i, (lo, hi, ln) in enumerate(self.groups):
            if lo <= b < hi:
                return i, ln
        return -1, 0

    def keys(self, b):
        """k, v [S][Hkv][D] in 64 bits: the group's prefix, then the sequence's own tokens."""
        g, _ = self.group(b)
        parts = ([self.rows[len(self.n) + g]] if g >= 0 else []) + [self.rows[b]]
        return [torch.cat([p[i] for p in parts]).double().cuda() for i in (0, 1)]


def attention_ref(bt, q, scale):
    """out [T][Hq][D], and per output the terms its error bound is made of: sum p|v|, the largest
    sum |q k| scale of a visible key, the number of visible keys, the largest visible |v|."""
    T, Hq, D = q.shape
    G = Hq // bt.Hkv
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    smax = torch.zeros((T, Hq, 1), dtype=torch.float64, device="cuda")
    cnt, vmax = (torch.zeros((T, 1, 1), dtype=torch.float64, device="cuda") for _ in range(2))
    for b, n in enumerate(bt.n):
        k, v = bt.keys(b)
        S = k.shape[0]
        for i in range(n):
            see = min(S, max(0, S - n + i + 1))
            if see == 0:
                continue
            t = bt.qs[b] + i
            qq = q[t].double().view(bt.Hkv, G, D)
            s = torch.einsum("hgd,shd->hgs", qq, k[:see]) * scale
            w = torch.softmax(s, -1)
            out[t] = torch.einsum("hgs,shd->hgd", w, v[:see]).reshape(Hq, D)
            mag[t] = torch.einsum("hgs,shd->hgd", w, v[:see].abs()).reshape(Hq, D)
            smax[t] = (torch.einsum("hgd,shd->hgs", qq.abs(), k[:see].abs()) * abs(scale)).amax(-1).view(Hq, 1)
            cnt[t] = see
            vmax[t] = v[:see].abs().amax()
    return out, mag, smax, cnt, vmax


def attention_tol(out, mag, smax, cnt, vmax, D, dtype, out_dtype):
    """|got - ref| bound.  A weight's relative error: its roundings for the tensor cores (half a
    step for one 16-bit term, half a step squared for two), the score's f32 sums (D/16 + 16
    additions of terms whose magnitudes sum to smax, each within 2^-23) and the exponential (2^-21);
    the sums over cnt keys: cnt/16 + 32 additions within 2^-23; f16 weights below 2^-14 of the
    largest keep steps of 2^-24 (half a step each); then the output's own rounding."""
    half = torch.finfo(DT[dtype]).eps / 2
    p = half * half if out_dtype == torch.float32 else half
    rel = p + (D / 16 + 16) * 2.0 ** -23 * smax + 2.0 ** -21 + (cnt / 16 + 32) * 2.0 ** -23
    tol = rel * mag + torch.finfo(out_dtype).eps / 2 * out.abs()
    if dtype == "f16":
        tol = tol + cnt * 2.0 ** -25 * vmax
    return tol + 1e-30


def rope_ref(x, pos, rot, theta, pairs):
    """x [T][H][D] in 64 bits, rotated at the positions."""
    y = x.clone()
    i = torch.arange(rot // 2, dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None, None] * theta ** (-2.0 * i / max(rot, 1))
    a = 2 * torch.arange(rot // 2, device=x.device) if pairs else torch.arange(rot // 2, device=x.device)
    b = a + 1 if pairs else a + rot // 2
    y[..., a] = x[..., a] * torch.cos(ang) - x[..., b] * torch.sin(ang)
    y[..., b] = x[..., a] * torch.sin(ang) + x[..., b] * torch.cos(ang)
    return y


def scale_of(D):
    return 1.0 / math.sqrt(D)
