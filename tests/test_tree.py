"""decode_attn_tree: nodes of trees of drafted tokens over the caches, against softmax
attention in fp64 straight from the definition.

Tolerance.  Scores are exact products (bf16, or f16 operands that hold the cache's
values) summed in fp32, and exponentials are off by about 2^-22: together they move a
weight by less than 2^-10 of itself here.  Weights enter the second product rounded once, by
at most half a bf16 step, 2^-8 of their size (f16: 2^-11), so that an output is off by at
most (2^-8 + 2^-10) sum_j p_j |v_j|; its own rounding adds 2^-8 of its magnitude.  f16
weights are formed 2^7 .. 2^15 at the largest and have an absolute step of 2^-24 at
the lower end, off by half of that: 2^-25 / 2^7 = 2^-32 of the largest weight, so of a sum that is
no smaller, for each entry (2^-32 sum_j |v_j|, quantized caches).  lse is
fp32: 1e-4, as for decode attention."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8 as OF
from oracle import nvfp4 as ON

gpu = pytest.mark.gpu
KV = ("bf16", "e4m3", "nvfp4")
K_SCALE, V_SCALE = 1.0 / 16, 1.0 / 24


@pytest.fixture(scope="module")
def api():
    from invariant_decode_attention_gb300 import api as _api
    _api.lib()
    return _api


def random_tree(rng, T):
    return [-1] + [int(rng.integers(max(-1, t - 5), t)) for t in range(1, T)]


def sees(parents, t, L, W, S, cap):
    """Entries that node t sees, from the definition."""
    def depth(a):
        return 0 if parents[a] < 0 else depth(parents[a]) + 1
    d = depth(t)
    got = [j for j in range(L) if W == 0 or j > L + d - W or j < S]
    a = t
    mine = []
    while a >= 0:
        e = depth(a)
        if W == 0 or d - e < W or L + e < S:
            mine.append(L + a)
        a = parents[a]
    return [j for j in got + sorted(mine) if j < cap]


class Case:
    def __init__(self, api, *, lengths, counts=None, T=4, heads=(8, 2, 128), layout="paged", kv="bf16", page=16,
                 window=0, sinks=0, tree=True, seed=0, room=0, q_gain=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        H_q, H, D = heads
        B = len(lengths)
        self.heads, self.layout, self.kv, self.page, self.T, self.B = heads, layout, kv, page, T, B
        self.window, self.sinks, self.lengths = window, sinks, list(lengths)
        self.counts = [T] * B if counts is None else list(counts)
        self.given_counts = counts is not None
        need = max(max(lengths) + T, 1) + room
        width = -(-need // page) if layout == "paged" else need
        if layout == "contiguous":
            blocks, total, self.table = 0, B * width, None
        else:
            blocks = B * width + 2
            total = blocks * (page if layout == "paged" else 1)
            self.table = torch.randperm(blocks, generator=g)[:B * width].view(B, width).int()
        self.width, self.total, self.blocks = width, total, blocks
        self.cap = width * page if layout == "paged" else width
        if kv == "bf16":
            self.kc, self.vc = (torch.randn((total, H, D), generator=g).bfloat16() for _ in range(2))
        elif kv == "e4m3":
            self.kc, self.vc = ((torch.randn((total, H, D), generator=g) * 16).to(torch.float8_e4m3fn).view(torch.uint8)
                                for _ in range(2))
        else:
            m = total * H * D
            self.kc, self.vc = (torch.cat([torch.randint(0, 256, (m // 2,), generator=g, dtype=torch.int32),
                                           torch.randint(56, 80, (m // 16,), generator=g, dtype=torch.int32)])
                                .to(torch.uint8) for _ in range(2))
        self.q = (torch.randn((B, T, H_q, D), generator=g) * q_gain).bfloat16()
        self.parents = [random_tree(rng, T) if tree else list(range(-1, T - 1)) for _ in range(B)]
        self.tree = tree
        self.scale = D ** -0.5
        self.prob = api.problem(batch=B, num_q_heads=H_q, num_kv_heads=H, head_dim_qk=D, layout=layout,
                                scale=self.scale, page_size=page if layout == "paged" else 0, width=width,
                                num_blocks=blocks, kv_dtype=KV.index(kv), k_scale=K_SCALE, v_scale=V_SCALE)

    def entry(self, b, j):
        if self.layout == "contiguous":
            return b * self.width + j
        if self.layout == "paged":
            return int(self.table[b, j // self.page]) * self.page + j % self.page
        return int(self.table[b, j])

    def values(self, cache, scale):
        """The whole cache in fp64."""
        H, D = self.heads[1:]
        if self.kv == "bf16":
            return cache.double().numpy()
        if self.kv == "e4m3":
            return OF.dequantize(cache.numpy(), scale)
        m = self.total * H * D
        c = cache.numpy()
        return ON.dequantize_cache(c[:m // 2].reshape(-1, H, D // 2), c[m // 2:].reshape(-1, H, D // 16), scale)

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def run(self, api, **kw):
        B, T, H_q, D = self.q.shape
        kw.setdefault("out", torch.full((B, T, H_q, D), 7.0, dtype=torch.bfloat16, device="cuda"))
        kw.setdefault("lse", torch.full((B, T, H_q), 7.0, device="cuda"))
        kw.setdefault("parents", self.i32(self.parents) if self.tree else None)
        kw.setdefault("counts", self.i32(self.counts) if self.given_counts else None)
        kw.setdefault("lengths", self.i32(self.lengths))
        kw.setdefault("table", None if self.table is None else self.table.cuda())
        lengths = kw.pop("lengths")
        k, v = kw.pop("caches", None) or (self.kc.cuda(), self.vc.cuda())
        return api.tree(self.prob, self.q.cuda(), k, v, lengths, window=self.window, sinks=self.sinks, **kw)

    def check(self, out, lse, rows=None):
        H_q, H, D = self.heads
        G = H_q // H
        k, v = self.values(self.kc, K_SCALE), self.values(self.vc, V_SCALE)
        out, lse, q = out.double().cpu().numpy(), lse.double().cpu().numpy(), self.q.double().numpy()
        for b in range(self.B) if rows is None else rows:
            n = max(0, min(self.counts[b], self.T))
            assert np.all(out[b, n:] == 7.0) and np.all(lse[b, n:] == 7.0)
            L = max(0, min(self.lengths[b], self.cap))
            for t in range(n):
                at = [self.entry(b, j) for j in sees(self.parents[b], t, L, self.window, self.sinks, self.cap)]
                if not at:
                    assert np.all(out[b, t] == 0) and np.all(np.isneginf(lse[b, t]))
                    continue
                for h in range(H):
                    s = self.scale * q[b, t, h * G:(h + 1) * G] @ k[at, h].T
                    m = s.max(-1, keepdims=True)
                    p = np.exp(s - m)
                    z = p.sum(-1, keepdims=True)
                    ref, mag = p @ v[at, h] / z, p @ np.abs(v[at, h]) / z
                    err = np.abs(out[b, t, h * G:(h + 1) * G] - ref)
                    tol = 1.25 * 2.0 ** -8 * mag + 2.0 ** -8 * np.abs(ref)
                    if self.kv != "bf16":
                        tol = tol + 2.0 ** -32 * np.abs(v[at, h]).sum(0)
                    assert np.all(err <= tol), (b, t, h, float((err / tol).max()))
                    assert np.all(np.abs(lse[b, t, h * G:(h + 1) * G] - (m + np.log(z))[:, 0]) <= 1e-4)


# (layout, kv, page, heads, T, lengths, counts, window, sinks, tree)
GRID = [
    ("paged", "bf16", 16, (8, 2, 128), 1, [0, 1, 63, 64, 700], None, 0, 0, False),
    ("paged", "bf16", 64, (32, 8, 128), 8, [130, 5, 0], [8, 3, 1], 0, 0, True),
    ("paged", "bf16", 32, (4, 4, 64), 64, [70, 0, 33], [64, 64, 1], 0, 0, True),
    ("contiguous", "bf16", 0, (16, 1, 128), 17, [200, 1, 64], [17, 0, 16], 0, 0, True),
    ("indexed", "bf16", 0, (7, 7, 128), 5, [77, 128, 3], None, 0, 0, True),
    ("paged", "bf16", 48, (24, 2, 64), 13, [500, 47, 48, 49], None, 0, 0, True),
    ("paged", "bf16", 3, (6, 2, 128), 9, [100, 2], None, 0, 0, True),
    ("paged", "bf16", 16, (128, 1, 128), 6, [300, 10], None, 0, 0, True),   # 768 rows: three units
    ("paged", "e4m3", 16, (20, 4, 64), 13, [333, 64, 0], [13, 7, 13], 0, 0, True),
    ("contiguous", "e4m3", 0, (32, 8, 128), 4, [129, 640], None, 0, 0, False),
    ("indexed", "e4m3", 0, (8, 1, 64), 33, [90], None, 0, 0, True),
    ("paged", "nvfp4", 16, (8, 1, 64), 7, [150, 31, 0], None, 0, 0, True),
    ("contiguous", "nvfp4", 0, (12, 3, 128), 21, [65, 200], [21, 20], 0, 0, True),
    ("indexed", "nvfp4", 0, (20, 4, 64), 3, [260], None, 0, 0, True),
    ("paged", "nvfp4", 1, (48, 2, 128), 6, [100, 7], None, 0, 0, True),
    # windows
    ("paged", "bf16", 16, (8, 2, 128), 1, [1000, 40, 0, 129], None, 128, 4, False),
    ("paged", "e4m3", 16, (8, 2, 128), 6, [2000, 333], None, 100, 70, True),
    ("contiguous", "bf16", 0, (8, 8, 64), 40, [500, 8], None, 7, 2, False),   # the window ends within the chain
    ("paged", "nvfp4", 64, (8, 2, 64), 30, [300, 2, 0], [30, 30, 29], 5, 4, True),
    ("indexed", "bf16", 0, (8, 2, 128), 4, [700], None, 1, 0, True),          # only itself
    ("paged", "bf16", 16, (8, 2, 128), 5, [600, 90], None, 200, 1000, True),  # sinks beyond the list
    ("paged", "bf16", 48, (8, 2, 128), 5, [900], None, 500, 129, True),
]


@gpu
@pytest.mark.parametrize("layout,kv,page,heads,T,lengths,counts,window,sinks,tree", GRID)
def test_against_definition(api, layout, kv, page, heads, T, lengths, counts, window, sinks, tree):
    c = Case(api, layout=layout, kv=kv, page=page, heads=heads, T=T, lengths=lengths, counts=counts, window=window,
             sinks=sinks, tree=tree, seed=T)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(api, err=err)
    assert int(err) == 0
    c.check(out, lse)


# (heads, T): (node, head) rows a KV head on both sides of every width that a kernel is made for
ROWS = [((7, 7, 128), 1), ((8, 1, 64), 1), ((32, 8, 128), 2), ((18, 2, 128), 1), ((32, 8, 128), 4), ((34, 2, 64), 1),
        ((24, 2, 128), 2), ((10, 2, 64), 5), ((15, 3, 128), 5), ((32, 8, 128), 8), ((16, 2, 64), 4), ((11, 1, 128), 3)]


@gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("heads,T", ROWS)
@pytest.mark.parametrize("layout,page,window", [("paged", 16, 0), ("paged", 5, 70), ("contiguous", 0, 300), ("indexed", 0, 0)])
def test_numbers_of_rows(api, kv, heads, T, layout, page, window):
    c = Case(api, kv=kv, heads=heads, T=T, layout=layout, page=page, lengths=[640, 5, 0, 61], window=window,
             sinks=5 if window else 0, tree=T > 2, seed=T + page)
    c.check(*c.run(api))


@gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("heads,T", [((8, 2, 64), 3), ((8, 8, 128), 2), ((32, 2, 128), 3)])
def test_layouts_give_the_same_bits(api, kv, heads, T):
    """Pages of 16 (copied whole), of 5 and single slots, and a contiguous cache."""
    H, D = heads[1:]
    L, rows = [700, 33], []
    base = Case(api, kv=kv, heads=heads, T=T, layout="contiguous", page=0, lengths=L, seed=21)
    for layout, page in (("contiguous", 0), ("paged", 16), ("paged", 5), ("indexed", 0)):
        c = Case(api, kv=kv, heads=heads, T=T, layout=layout, page=page, lengths=L, seed=21)
        c.q, c.parents = base.q, base.parents
        for b in range(2):
            for j in range(L[b] + T):
                to, at = c.entry(b, j), base.entry(b, j)
                for mine, its in ((c.kc, base.kc), (c.vc, base.vc)):
                    if kv != "nvfp4":
                        mine[to] = its[at]
                        continue
                    m, m0 = c.total * H * D // 2, base.total * H * D // 2
                    mine[:m].view(-1, H * D // 2)[to] = its[:m0].view(-1, H * D // 2)[at]
                    mine[m:].view(-1, H * D // 16)[to] = its[m0:].view(-1, H * D // 16)[at]
        rows.append(c.run(api))
    for out, lse in rows[1:]:
        assert torch.equal(out, rows[0][0]) and torch.equal(lse, rows[0][1])


@gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("heads,T", [((8, 8, 128), 4), ((8, 2, 64), 4), ((48, 2, 128), 1)])
def test_a_short_row_depends_on_itself_alone(api, kv, heads, T):
    """Rows of few nodes, alone and in batches of any size and order, and again."""
    rng = np.random.default_rng(22)
    lengths = [int(x) for x in rng.integers(0, 2500, 40)]
    counts = [int(x) for x in rng.integers(1, T + 1, 40)]
    c = Case(api, kv=kv, heads=heads, T=T, lengths=lengths, counts=counts, window=900, sinks=2, seed=22)
    out, lse = c.run(api)
    again = c.run(api)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    q, table, parents = c.q.clone(), c.table.clone(), list(c.parents)
    for rows in ([7], [39, 0], [int(x) for x in rng.permutation(40)], [5] * 3):
        c.prob.batch = c.B = len(rows)
        c.q, c.table, c.parents = q[rows], table[rows].contiguous(), [parents[b] for b in rows]
        c.lengths, c.counts = [lengths[b] for b in rows], [counts[b] for b in rows]
        got = c.run(api)
        assert torch.equal(got[0], out[rows]) and torch.equal(got[1], lse[rows])


@gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("heads", [(8, 2, 64), (16, 2, 64)])  # 24 rows a KV head, 48: the two kernels
def test_peaked_scores(api, kv, heads):
    # large scores: the running reference value moves many times
    c = Case(api, kv=kv, T=6, lengths=[1500, 700], heads=heads, q_gain=12.0, seed=3)
    c.check(*c.run(api))


@gpu
@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_other_scales(api, scale):
    c = Case(api, T=3, lengths=[400, 9], seed=4)
    c.scale = c.prob.scale = scale
    c.check(*c.run(api))


@gpu
@pytest.mark.parametrize("kv,heads", [("bf16", (32, 8, 128)), ("e4m3", (8, 2, 64)), ("nvfp4", (16, 2, 128))])
def test_long_rows_have_many_splits(api, kv, heads):
    c = Case(api, kv=kv, heads=heads, T=5, lengths=[9000, 513, 512, 2047], page=64, seed=5)
    c.check(*c.run(api))


@gpu
def test_a_row_depends_on_itself_alone(api):
    """Alone, in any batch and position, with room for more nodes, under other page ids."""
    heads, n, L = (16, 4, 128), 11, 1300
    base = Case(api, heads=heads, T=n, lengths=[L], seed=6)
    alone = [x[0] for x in base.run(api)]
    rng = np.random.default_rng(6)
    H_q, H, D = heads
    for B, T in ((3, 11), (40, 16), (7, 64)):
        lengths = [int(x) for x in rng.integers(0, 3000, B)]
        counts = [int(x) for x in rng.integers(0, T + 1, B)]
        b = int(rng.integers(B))
        lengths[b], counts[b] = L, n
        c = Case(api, heads=heads, T=T, lengths=lengths, counts=counts, seed=B)
        c.parents[b][:n] = base.parents[0]
        c.q[b, :n] = base.q[0]
        for j in range(L + n):
            c.kc[c.entry(b, j)], c.vc[c.entry(b, j)] = base.kc[base.entry(0, j)], base.vc[base.entry(0, j)]
        out, lse = c.run(api)
        assert torch.equal(out[b, :n], alone[0]) and torch.equal(lse[b, :n], alone[1])
        again = c.run(api)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@gpu
def test_more_rows_than_a_launch_takes(api):
    lengths = [int(x) for x in np.random.default_rng(8).integers(0, 90, 2100)]
    c = Case(api, heads=(2, 1, 64), T=2, lengths=lengths, seed=8)
    c.check(*c.run(api), rows=[0, 1, 1023, 1024, 1500, 2047, 2048, 2099])


@gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("heads", [(8, 2, 64), (16, 2, 64), (2, 2, 128)])
def test_what_lies_in_unseen_places_does_not_matter(api, kv, window, heads):
    """NaN (and for bf16 infinities) past the end, in the window's hole, in pages of nobody,
    and in a sibling's entry, whose K and V only that node sees."""
    L, T = 1000, 6
    c = Case(api, kv=kv, T=T, lengths=[L, 30], heads=heads, window=window, sinks=3 if window else 0, seed=9, room=70)
    c.parents = [[-1, 0, 0, 2, 2, -1]] * 2  # node 1 is seen by itself alone
    clean = c.run(api)
    c.check(*clean)
    H, D = c.heads[1:]
    seen = {c.entry(b, j) for b in range(2) for t in range(T) if t != 1
            for j in sees(c.parents[b], t, c.lengths[b], window, c.sinks, c.cap)}
    spoil = torch.tensor([e for e in range(c.total) if e not in seen])
    was = c.kc.clone(), c.vc.clone()
    for cache in (c.kc, c.vc):
        if kv == "bf16":
            cache[spoil] = float("nan")
            cache[spoil[::3]] = float("inf")
        elif kv == "e4m3":
            cache[spoil] = 0x7f
        else:
            m = c.total * H * D
            cache[m // 2:].view(-1, H, D // 16)[spoil] = 0x7f
    out, lse = c.run(api)
    keep = [0, 2, 3, 4, 5]
    assert torch.isfinite(out[:, keep].float()).all() and torch.isfinite(lse[:, keep]).all()
    assert out[:, 1].isnan().all() and lse[:, 1].isnan().all()
    c.kc, c.vc = was
    out[:, 1], lse[:, 1] = clean[0][:, 1], clean[1][:, 1]
    c.check(out, lse)


@gpu
def test_nan_and_infinity_in_seen_places(api):
    c = Case(api, T=4, lengths=[200], heads=(4, 2, 64), seed=10)
    c.parents = [[-1, 0, 1, -1]]
    c.kc[c.entry(0, 201), 0] = float("nan")   # node 1, seen by 1 and 2, KV head 0
    c.vc[c.entry(0, 203), 1, 5] = float("inf")  # node 3, seen by itself, KV head 1
    out, lse = c.run(api)
    out, lse = out.float().cpu(), lse.cpu()
    assert out[0, 1:3, :2].isnan().all() and lse[0, 1:3, :2].isnan().all()
    assert torch.isfinite(out[0, :3, 2:]).all() and torch.isfinite(out[0, [0, 3], :2]).all()
    assert torch.isposinf(out[0, 3, 2:, 5]).all()
    rest = [d for d in range(64) if d != 5]
    assert torch.isfinite(out[0, 3, 2:][:, rest]).all() and torch.isfinite(lse[0, 3, 2:]).all()


@gpu
def test_bits_of_bad_input(api):
    def bits(c, **kw):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        r = c.run(api, err=err, **kw)
        return int(err), r

    c = Case(api, T=3, lengths=[60, 100, 20], seed=11)
    code, _ = bits(c)
    assert code == 0
    # lengths and counts out of range are clamped, other rows are as ever
    c.lengths = [60, -5, 20]
    code, r = bits(c)
    assert code == api.DEVERR_LENGTH
    c.check(*r)
    c.lengths = [60, c.cap + 9, 20]  # the nodes' own entries lie beyond the capacity
    code, r = bits(c)
    assert code == api.DEVERR_LENGTH
    c.check(*r)
    c.lengths, c.counts, c.given_counts = [60, c.cap - 2, 20], [3, 3, 3], True
    code, r = bits(c)
    assert code == api.DEVERR_LENGTH
    c.check(*r)
    c.lengths, c.counts = [60, 100, 20], [3, 77, -1]
    code, r = bits(c)
    assert code == api.DEVERR_LENGTH
    c.check(*r)
    # parents that are no earlier nodes count as none
    c.counts = [3, 3, 3]
    c.parents[1] = [-1, 1, -2]
    code, r = bits(c)
    assert code == api.DEVERR_INDEX
    c.parents[1] = [-1, -1, -1]
    c.check(*r)
    # a page out of range: only where some node sees an entry of it
    for bad in (-1, c.blocks):
        t = c.table.clone()
        t[1, 2] = bad
        code, r = bits(c, table=t.cuda())
        assert code == api.DEVERR_INDEX
        c.check(*r, rows=[0, 2])
        c.window, c.sinks = 40, 16
        t = c.table.clone()
        t[1, 1:3] = bad  # entries 16 .. 47 of 100: in the window's hole
        code, r = bits(c, table=t.cuda())
        assert code == 0
        c.check(*r)
        c.window = c.sinks = 0
        t = c.table.clone()
        t[0, 4:] = bad  # behind the row's end
        t[2, 2:] = bad
        code, r = bits(c, table=t.cuda())
        assert code == 0
        c.check(*r)


@gpu
def test_a_row_of_capacity_zero(api):
    c = Case(api, layout="contiguous", T=2, lengths=[5], seed=12)
    c.prob.width = 0
    nothing = torch.zeros(8, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(api, err=err, caches=(nothing, nothing.clone()))
    assert int(err) == api.DEVERR_LENGTH
    assert (out == 0).all() and torch.isneginf(lse).all()


@gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("heads,T", [((32, 32, 64), 1), ((64, 32, 128), 3), ((128, 32, 64), 5), ((96, 8, 64), 4)])
def test_rows_without_a_tile_among_others(api, kv, heads, T):
    """Full rows with a window of one: their nodes see nothing.  A block has a dozen units
    of such rows one after another, and some of rows that see something."""
    lengths = [64] * 300
    for b, L in ((0, 63), (100, 0), (199, 5), (200, 63), (254, 17), (255, 1), (299, 40)):
        lengths[b] = L
    c = Case(api, kv=kv, heads=heads, T=T, layout="contiguous", page=0, lengths=lengths, window=1, room=-T, seed=18)
    assert c.cap == 64
    c.lengths[7] = c.lengths[201] = 99  # clamped
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(api, err=err)
    assert int(err) == api.DEVERR_LENGTH
    c.check(out, lse)
    # all rows of a call
    c.lengths = [64] * 300
    out, lse = c.run(api)
    assert (out == 0).all() and torch.isneginf(lse).all()
    # and with places left for more nodes
    c.lengths, c.counts, c.given_counts = list(lengths), [b % (T + 1) for b in range(300)], True
    c.check(*c.run(api))


@gpu
def test_streams_and_graphs(api):
    a = Case(api, T=5, lengths=[900, 20], seed=13)
    b = Case(api, T=7, lengths=[40, 1500, 3], kv="e4m3", window=64, sinks=4, seed=14)
    want = [c.run(api) for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        got = [c.run(api, stream=s) for c, s in zip((a, b), streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])
    # captured and replayed with other contents: lengths, tree and queries are read on the device
    q, lengths, parents = a.q.cuda(), a.i32(a.lengths), a.i32(a.parents)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    ws, k, v, table = api.tree_workspace(a.prob, 5), a.kc.cuda(), a.vc.cuda(), a.table.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.tree(a.prob, q, k, v, lengths, parents=parents, table=table, out=out, lse=lse, ws=ws)
    graph.replay()
    assert torch.equal(out, want[0][0]) and torch.equal(lse, want[0][1])
    a.lengths, a.parents = [17, 600], [[-1, 0, 0, 1, 1], [-1, -1, 1, 2, 0]]
    a.q = torch.randn_like(a.q.float()).bfloat16()
    q.copy_(a.q)
    lengths.copy_(a.i32(a.lengths))
    parents.copy_(a.i32(a.parents))
    graph.replay()
    a.check(out, lse)


@gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("heads", [(8, 2, 128), (32, 2, 128)])
def test_time_out_path(api, kv, heads):
    c = Case(api, kv=kv, T=4, lengths=[700, 90], heads=heads, seed=15)
    want = c.run(api)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.prob.flags = api.FLAG_TEST_STALL
    for _ in range(2):
        err.zero_()
        c.run(api, err=err)
        assert int(err) == api.DEVERR_TIMEOUT
    c.prob.flags = 0
    err.zero_()
    got = c.run(api, err=err)
    assert int(err) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("layout,page", [("paged", 16), ("contiguous", 0)])
@pytest.mark.parametrize("T", [1, 5])
def test_time_out_with_copies_on_their_way(api, kv, layout, page, T):
    """Few rows, entries copied in boxes: every wait for one runs out, in blocks that have
    several units each.  Other calls beside it and after it are as ever."""
    rng = np.random.default_rng(23)
    c = Case(api, kv=kv, T=T, lengths=[int(x) for x in rng.integers(0, 1500, 200)], heads=(16, 4, 128), layout=layout,
             page=page, seed=23)
    b = Case(api, kv=kv, T=T, lengths=[1100, 30, 400], heads=(16, 4, 128), layout=layout, page=page, seed=24)
    want = [x.run(api) for x in (c, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    inputs = [(x.prob, x.q.cuda(), x.kc.cuda(), x.vc.cuda(), x.i32(x.lengths)) for x in (c, b)]
    more = [dict(parents=x.i32(x.parents), table=None if x.table is None else x.table.cuda(), ws=api.tree_workspace(x.prob, T))
            for x in (c, b)]
    for _ in range(3):
        err, none = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
        outs = [(torch.full_like(inputs[i][1], 7.0), torch.full(inputs[i][1].shape[:3], 7.0, device="cuda"))
                for i in (0, 0, 1, 1, 1)]
        torch.cuda.synchronize()
        c.prob.flags = api.FLAG_TEST_STALL
        api.tree(*inputs[0], **more[0], out=outs[0][0], lse=outs[0][1], err=err, stream=streams[0])
        c.prob.flags = 0
        for out, lse in outs[2:]:
            api.tree(*inputs[1], **more[1], out=out, lse=lse, err=none, stream=streams[1])
        api.tree(*inputs[0], **more[0], out=outs[1][0], lse=outs[1][1], err=none, stream=streams[0])
        torch.cuda.synchronize()
        assert int(err) == api.DEVERR_TIMEOUT and int(none) == 0
        assert (outs[0][0] != 7.0).any()  # the units were gone through
        for i, (out, lse) in zip((0, 1, 1, 1), outs[1:]):
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


@gpu
@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("H_q,T", [(8, 3), (128, 3)])
def test_caches_beyond_32_bits(api, kv, H_q, T):
    """A cache of more than 2^32 elements, pages at both ends of it and around 2^31 and 2^32."""
    H, D, page = 8, 128, 16
    pages = (1 << 18) + 7  # 16384 elements each
    c = Case(api, kv=kv, heads=(H_q, H, D), T=T, lengths=[120], page=page, seed=16)
    small = c.run(api)
    ids = [0, (1 << 17) - 1, 1 << 17, (1 << 18) - 1, 1 << 18, pages - 2, pages - 1, 77]
    n = c.width
    assert n == len(ids)
    rows = torch.tensor([[i * page + j for j in range(page)] for i in ids]).view(-1)
    old = torch.tensor([[int(c.table[0, i]) * page + j for j in range(page)] for i in range(n)]).view(-1)
    big = []
    for cache in (c.kc, c.vc):
        m, s = pages * page * H * D, c.total * H * D
        if kv == "nvfp4":
            t = torch.zeros(m // 2 + m // 16, dtype=torch.uint8, device="cuda")
            t[:m // 2].view(-1, H * D // 2)[rows.cuda()] = cache[:s // 2].view(-1, H * D // 2)[old].cuda()
            t[m // 2:].view(-1, H * D // 16)[rows.cuda()] = cache[s // 2:].view(-1, H * D // 16)[old].cuda()
        else:
            t = torch.zeros((pages * page, H, D), dtype=cache.dtype, device="cuda")
            t[rows.cuda()] = cache[old].cuda()
        big.append(t)
    c.prob.num_blocks = pages
    got = c.run(api, caches=big, table=c.i32([ids]))
    assert torch.equal(got[0], small[0]) and torch.equal(got[1], small[1])
    del big, t
    torch.cuda.empty_cache()


@gpu
@pytest.mark.parametrize("kv", KV)
def test_one_node_is_decode_attention(api, kv):
    """Without a window, a row's single node attends as the next token of a plain step."""
    c = Case(api, kv=kv, heads=(8, 2, 128), T=1, lengths=[0, 17, 300, 1100], seed=17)
    out, lse = c.run(api)
    ws = api.workspace(c.prob)
    o2, l2 = torch.empty_like(out[:, 0]), torch.empty_like(lse[:, 0])
    api.forward(c.prob, api.INVARIANT, c.q[:, 0].contiguous().cuda(), c.kc.cuda(), c.vc.cuda(), c.table.cuda(),
                c.i32([x + 1 for x in c.lengths]), ws, o2, l2)
    assert float((out[:, 0].float() - o2.float()).abs().max()) <= 2e-2
    assert float((lse[:, 0] - l2).abs().max()) <= 2e-4


# ------------------------------------------------------------------ refusals (CPU)

def fake_args(api, prob, **kw):
    size = ctypes.c_size_t()
    ok = api.lib().decode_attn_tree_workspace_bytes(ctypes.byref(prob), 4, ctypes.byref(size)) == 0
    a = dict(nodes=4, window=0, sinks=0, parents=0, counts=0, q=1 << 20, k=1 << 21, v=1 << 22, table=1 << 23,
             lengths=1 << 24, out=1 << 26, lse=1 << 28, err=0, ws=1 << 30, ws_bytes=size.value if ok else 0)
    a.update(kw)
    return api._TREE.pack(*(a[k] for k in ("nodes", "window", "sinks", "parents", "counts", "q", "k", "v", "table",
                                           "lengths", "out", "lse", "err", "ws", "ws_bytes")))


def small_problem(api, **kw):
    args = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim_qk=128, layout="paged", scale=0.1, page_size=16,
                width=64, num_blocks=200)
    args.update(kw)
    return api.problem(**args)


def call(api, prob, **kw):
    return api.lib().decode_attn_tree(ctypes.addressof(prob), fake_args(api, prob, **kw), None)


def test_argument_rules(api):
    p = small_problem(api)
    inv, uns, wsp = api.ERR_INVALID_ARG, api.ERR_UNSUPPORTED, api.ERR_WORKSPACE
    assert api.lib().decode_attn_tree(None, fake_args(api, p), None) == inv
    assert api.lib().decode_attn_tree(ctypes.addressof(p), None, None) == inv
    for kw in (dict(nodes=0), dict(nodes=-1), dict(window=-1), dict(sinks=-1), dict(q=0), dict(k=0), dict(v=0),
               dict(lengths=0), dict(out=0), dict(lse=0), dict(table=0), dict(q=(1 << 20) + 8), dict(k=(1 << 21) + 8),
               dict(out=(1 << 26) + 4), dict(lse=(1 << 28) + 2), dict(parents=2), dict(counts=(1 << 12) + 1),
               dict(err=(1 << 12) + 1), dict(lengths=(1 << 24) + 2), dict(out=1 << 20), dict(lse=(1 << 20) + 4),
               dict(lse=(1 << 26) + 64)):
        assert call(api, p, **kw) == inv, kw
    # outputs over what other blocks read or write meanwhile
    out, lse = 1 << 26, 1 << 28
    for kw in (dict(lengths=out + 64), dict(counts=lse + 8), dict(parents=out + 128), dict(table=lse + 16),
               dict(k=out), dict(v=out + 4096), dict(k=lse), dict(ws=out), dict(ws=lse)):
        assert call(api, p, **kw) == inv, kw
    assert call(api, p, nodes=65) == uns
    need = api.tree_workspace_bytes(p, 4)
    for kw in (dict(ws=0), dict(ws=(1 << 30) + 16), dict(ws_bytes=need - 1)):
        assert call(api, p, **kw) == wsp, kw
    flat = small_problem(api, layout="contiguous", page_size=0, num_blocks=0)
    assert call(api, flat) == inv  # a contiguous cache has no table
    for kw in (dict(head_dim_qk=96), dict(head_dim_qk=576, head_dim_v=512, num_kv_heads=1, num_q_heads=16,
                                          shared_latent=True), dict(num_q_heads=258, num_kv_heads=2),
               dict(extra_width=4, extra_num_blocks=9), dict(head_dim_v=64), dict(num_blocks=1 << 27)):
        assert call(api, small_problem(api, **kw)) == uns, kw
    assert call(api, small_problem(api, scale=float("nan"))) == inv
    assert call(api, small_problem(api, batch=0)) == api.OK  # nothing to do, nothing is looked at


def test_workspace_sizes(api):
    p = small_problem(api)
    assert api.tree_workspace_bytes(p, 4) >= 2 * 2 * 4 * 8 * (128 + 1) * 4
    short = small_problem(api, width=8)  # 128 entries: one split
    assert api.tree_workspace_bytes(short, 64) == 256
    n = ctypes.c_size_t()
    L = api.lib()
    assert L.decode_attn_tree_workspace_bytes(ctypes.byref(p), 65, ctypes.byref(n)) == api.ERR_UNSUPPORTED
    assert L.decode_attn_tree_workspace_bytes(ctypes.byref(p), 0, ctypes.byref(n)) == api.ERR_INVALID_ARG
    assert L.decode_attn_tree_workspace_bytes(ctypes.byref(p), 4, None) == api.ERR_INVALID_ARG


def test_python_checks(api):
    p = small_problem(api)
    q = torch.zeros((2, 4, 8, 128), dtype=torch.bfloat16)
    k = torch.zeros((200, 16, 2, 128), dtype=torch.bfloat16)
    lengths, table = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 64), dtype=torch.int32)
    out, lse, ws = torch.zeros_like(q), torch.zeros((2, 4, 8)), torch.zeros(1 << 24, dtype=torch.uint8)
    ok = dict(table=table, out=out, lse=lse, ws=ws)
    with pytest.raises(ValueError, match="no CPU path"):
        api.tree(p, q, k, k.clone(), lengths, **ok)
    for kw, word in ((dict(table=None), "table"), (dict(table=table[:1]), "table"), (dict(out=out[:, :3]), "out"),
                     (dict(lse=lse.double()), "lse"), (dict(counts=lengths.long()), "counts"),
                     (dict(parents=torch.zeros((2, 3), dtype=torch.int32)), "parents")):
        with pytest.raises(ValueError, match=word):
            api.tree(p, q, k, k.clone(), lengths, **{**ok, **kw})
    with pytest.raises(ValueError, match="separate"):
        api.tree(p, q, k, None, lengths, **ok)
    with pytest.raises(ValueError, match="k holds"):
        api.tree(p, q, k[:100], k, lengths, **ok)
    with pytest.raises(ValueError, match="q must"):
        api.tree(p, q.float(), k, k.clone(), lengths, **ok)
    with pytest.raises(ValueError, match="q must"):
        api.tree(p, q[:1], k, k.clone(), lengths, **ok)


def test_the_definition_used_here():
    # hand-worked: context of 3, a tree 0 <- 1, 0 <- 2 <- 3
    par = [-1, 0, 0, 2]
    assert sees(par, 3, 3, 0, 0, 99) == [0, 1, 2, 3, 5, 6]
    assert sees(par, 1, 3, 0, 0, 99) == [0, 1, 2, 3, 4]
    assert sees(par, 3, 3, 2, 0, 99) == [5, 6]        # position 5 sees 4 and 5
    assert sees(par, 3, 3, 4, 0, 99) == [2, 3, 5, 6]  # positions 2 .. 5
    assert sees(par, 3, 3, 2, 1, 99) == [0, 5, 6]
    assert sees(par, 3, 0, 2, 1, 99) == [0, 2, 3]     # the root is the first position
    assert sees(par, 3, 3, 0, 0, 6) == [0, 1, 2, 3, 5]
