"""decode_attn_copy_pages and decode_attn_compact: bytes of the caches of all layers
against the same moves in numpy, bit for bit."""

import ctypes

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
KV = ("bf16", "e4m3", "nvfp4")


@pytest.fixture(scope="module")
def api():
    from invariant_decode_attention_gb300 import api as _api
    _api.lib()
    return _api


class Case:
    def __init__(self, api, *, layout="paged", kv="bf16", heads=2, D=128, page=16, layers=3, B=4, width=6, latent=False,
                 seed=0):
        g = torch.Generator().manual_seed(seed)
        self.layout, self.kv, self.page, self.B, self.width, self.layers = layout, kv, page, B, width, layers
        pages = B * width + 3
        self.table = None
        if layout == "contiguous":
            self.total, self.cap, blocks = B * width, width, 0
        else:
            self.total = pages * (page if layout == "paged" else 1)
            self.cap, blocks = width * (page if layout == "paged" else 1), pages
            self.table = torch.randperm(pages, generator=g)[:B * width].view(B, width).int()
        self.blocks = blocks
        self.prob = api.problem(batch=B, num_q_heads=16 if latent else heads, num_kv_heads=1 if latent else heads,
                                head_dim_qk=D, head_dim_v=512 if latent else D, layout=layout, scale=0.1,
                                page_size=page if layout == "paged" else 0, width=width, num_blocks=blocks,
                                kv_dtype=KV.index(kv), shared_latent=latent)
        m = self.total * heads * D
        size = {"bf16": 2 * m, "e4m3": m, "nvfp4": m // 2 + m // 16}[kv]
        self.cut = [(0, size, size // self.total)] if kv != "nvfp4" else [
            (0, m // 2, heads * D // 2), (m // 2, size, heads * D // 16)]  # from, to, bytes of an entry
        self.bytes = [torch.randint(0, 256, (size,), generator=g, dtype=torch.int32).to(torch.uint8).cuda()
                      for _ in range(layers * (1 if latent else 2))]
        self.before = [t.cpu().numpy() for t in self.bytes]
        t = [x.view(torch.bfloat16) if kv == "bf16" else x for x in self.bytes]
        self.caches = api.Caches(self.prob, t[:layers], None if latent else t[layers:])

    def entry(self, b, j):
        if self.layout == "contiguous":
            return b * self.width + j
        if self.layout == "paged":
            return int(self.table[b, j // self.page]) * self.page + j % self.page
        return int(self.table[b, j])

    def check(self, moves):
        """moves: (from, to) entries, all read before any is written."""
        for now, was in zip(self.bytes, self.before):
            want = was.copy()
            for lo, hi, size in self.cut:
                a, b = want[lo:hi].reshape(-1, size), was[lo:hi].reshape(-1, size)
                for i, j in moves:
                    a[j] = b[i]
            assert np.array_equal(now.cpu().numpy(), want)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ pages

@gpu
@pytest.mark.parametrize("layout,kv,heads,D,page,latent", [
    ("paged", "bf16", 2, 128, 16, False), ("paged", "bf16", 8, 128, 64, False), ("paged", "e4m3", 1, 64, 1, False),
    ("paged", "nvfp4", 1, 64, 1, False), ("paged", "nvfp4", 3, 64, 3, False), ("paged", "nvfp4", 8, 128, 48, False),
    ("indexed", "bf16", 2, 64, 0, False), ("indexed", "nvfp4", 1, 128, 0, False), ("paged", "bf16", 1, 576, 16, True),
    ("indexed", "e4m3", 1, 576, 0, True)])
def test_copies(api, layout, kv, heads, D, page, latent):
    c = Case(api, layout=layout, kv=kv, heads=heads, D=D, page=page, latent=latent, seed=page + D)
    src, dst = [5, 5, 7, -1, 9, 11, 2, 26], [0, 1, 3, 4, 9, -3, 8, 10]  # 5 twice, nothing, itself, nothing
    err = i32([0])
    api.copy_pages(c.prob, c.caches, i32(src), i32(dst), err=err)
    assert int(err) == 0
    per = page if layout == "paged" else 1
    c.check([(s * per + e, d * per + e) for s, d in zip(src, dst) if s >= 0 and d >= 0 for e in range(per)])


@gpu
def test_many_layers_and_pairs(api):
    c = Case(api, layers=70, B=20, width=4, heads=1, D=64, page=2, seed=1)  # 140 buffers: two launches
    src, dst = list(range(0, 40)), list(range(40, 80))
    api.copy_pages(c.prob, c.caches, i32(src), i32(dst))
    c.check([(s * 2 + e, d * 2 + e) for s, d in zip(src, dst) for e in range(2)])
    big = Case(api, layers=1, B=1, width=140000, heads=1, D=64, page=1, kv="e4m3", seed=2)
    n = 70000  # more pairs than a grid's second dimension
    api.copy_pages(big.prob, big.caches, torch.arange(n, **dict(dtype=torch.int32, device="cuda")),
                   torch.arange(n, 2 * n, **dict(dtype=torch.int32, device="cuda")))
    for now, was in zip(big.bytes, big.before):
        want = was.reshape(-1, 64).copy()
        want[n:2 * n] = want[:n]
        assert np.array_equal(now.cpu().numpy().reshape(-1, 64), want)


@gpu
def test_pages_out_of_range(api):
    c = Case(api, seed=3)
    err = i32([0])
    api.copy_pages(c.prob, c.caches, i32([0, c.blocks, 1]), i32([c.blocks + 5, 3, 4]), err=err)
    assert int(err) == api.DEVERR_INDEX
    c.check([(16 + e, 64 + e) for e in range(16)])
    api.copy_pages(c.prob, c.caches, i32([c.blocks]), i32([0]))  # not reported, not done either
    c.check([(16 + e, 64 + e) for e in range(16)])
    api.copy_pages(c.prob, c.caches, i32([]), i32([]))


@gpu
@pytest.mark.parametrize("kv", ["e4m3", "nvfp4"])
def test_caches_beyond_32_bits(api, kv):
    """Pages and entries on both sides of 2^31 and 2^32 bytes of a buffer, block scales behind them."""
    heads, D, page, pages = 8, 128, 64, (1 << 18) + 9  # 64 KB of elements a page
    per = heads * D * page
    prob = api.problem(batch=1, num_q_heads=heads, num_kv_heads=heads, head_dim_qk=D, layout="paged", scale=0.1,
                       page_size=page, width=2, num_blocks=pages, kv_dtype=KV.index(kv))
    m = pages * per
    size = m if kv == "e4m3" else m // 2 + m // 16
    k, v = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    caches = api.Caches(prob, [k], [v])
    # (parts: elements or codes, block scales)
    parts = [(0, m, per)] if kv == "e4m3" else [(0, m // 2, per // 2), (m // 2, size, per // 16)]
    g = torch.Generator().manual_seed(24)
    ends = [0, (1 << 15) - 1, 1 << 15, (1 << 16) - 1, 1 << 16, (1 << 17) - 1, 1 << 17, pages - 9]
    to = [pages - 1 - i for i in range(4)] + [1, 2, 3, 4]
    filled = {}
    for which, cache in enumerate((k, v)):
        for lo, hi, n in parts:
            for i in ends:
                filled[which, lo, i] = torch.randint(0, 256, (n,), generator=g, dtype=torch.int32).to(torch.uint8).cuda()
                cache[lo:hi].view(-1, n)[i] = filled[which, lo, i]
    api.copy_pages(prob, caches, i32(ends), i32(to))
    # entries 62 to 66 of a row over the last page and one at 2^32 bytes or past it: nodes 0, 2 and 4 of 62 stand
    row = [pages - 1, 1 << 16]
    new = api.compact(prob, caches, i32([62]), i32([[0, 2, 4, -1, -1]]), i32([2]), table=i32([row]))
    assert new.tolist() == [65]
    for which, cache in enumerate((k, v)):
        for lo, hi, n in parts:
            now = cache[lo:hi].view(-1, n)
            last, next_ = filled[which, lo, ends[0]].view(page, -1).clone(), filled[which, lo, 1 << 16].view(page, -1).clone()
            last[63] = next_[0]
            next_[0] = next_[2]
            assert torch.equal(now[row[0]].view(page, -1), last) and torch.equal(now[row[1]].view(page, -1), next_)
            for i, j in list(zip(ends, to))[1:]:
                assert torch.equal(now[j], filled[which, lo, i])
    del k, v, caches, cache, now
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ accepted entries

def paths(rng, B, T):
    """Ascending node lists, padded with -1, and accepted counts."""
    nodes, accepted = np.full((B, T), -1), rng.integers(0, T, B)
    for b in range(B):
        nodes[b, :accepted[b] + 1] = np.concatenate([[0], np.sort(rng.choice(np.arange(1, T), accepted[b], replace=False))])
    return nodes, accepted


@gpu
@pytest.mark.parametrize("layout,kv,heads,D,page,T,latent", [
    ("paged", "bf16", 2, 128, 16, 8, False), ("paged", "bf16", 8, 128, 4, 20, False), ("contiguous", "bf16", 2, 64, 0, 64, False),
    ("indexed", "e4m3", 1, 64, 0, 7, False), ("paged", "nvfp4", 1, 64, 3, 11, False), ("contiguous", "nvfp4", 20, 128, 0, 64, False),
    ("paged", "e4m3", 5, 64, 16, 1, False), ("paged", "bf16", 1, 576, 16, 33, True)])
def test_compaction(api, layout, kv, heads, D, page, T, latent):
    rng = np.random.default_rng(T)
    width = {"paged": -(-(T + 30) // max(page, 1))}.get(layout, T + 30)
    c = Case(api, layout=layout, kv=kv, heads=heads, D=D, page=page, width=width, B=9, latent=latent, seed=T)
    nodes, accepted = paths(rng, 9, T)
    lengths = rng.integers(0, 31, 9)
    nodes[4] = -1  # no nodes
    accepted[4] = 0
    err = i32([0])
    new = api.compact(c.prob, c.caches, i32(lengths), i32(nodes), i32(accepted),
                      table=None if c.table is None else c.table.cuda(), err=err)
    assert int(err) == 0
    kept = np.where(np.arange(9) == 4, 0, accepted + 1)
    assert new.tolist() == (lengths + kept).tolist()
    c.check([(c.entry(b, lengths[b] + nodes[b, i]), c.entry(b, lengths[b] + i)) for b in range(9) for i in range(kept[b])])


@gpu
def test_the_longest_shift(api):
    # every node but the second: each of 62 entries moves into the place of the one before it
    c = Case(api, width=8, B=1, seed=5)
    nodes = [[0] + list(range(2, 64)) + [-1]]
    api.compact(c.prob, c.caches, i32([50]), i32(nodes), i32([62]), table=c.table.cuda())
    c.check([(c.entry(0, 50 + n), c.entry(0, 50 + i)) for i, n in enumerate(nodes[0][:63])])


@gpu
def test_bad_rows_are_left(api):
    c = Case(api, B=8, width=6, seed=6)  # 96 entries a row
    T = 6
    good = [0, 2, 5, -1, -1, -1]
    nodes = [list(good) for _ in range(8)]
    accepted, lengths = [2] * 8, [10] * 8
    table = c.table.clone()
    nodes[1] = [0, 5, 2, -1, -1, -1]  # not ascending
    nodes[2] = [0, 2, 6, -1, -1, -1]  # no such node
    accepted[3] = 6
    accepted[4] = -1
    lengths[5] = 93                   # entry 98 lies beyond the capacity
    table[6, 0] = c.blocks            # the page of entries 10 .. 15
    err = i32([0])
    args = dict(table=table.cuda(), err=err)
    new = api.compact(c.prob, c.caches, i32(lengths), i32(nodes), i32(accepted), **args)
    assert int(err) == api.DEVERR_LENGTH | api.DEVERR_INDEX
    assert new.tolist() == [13, 10, 10, 10, 10, 93, 10, 13]
    done = [(c.entry(b, 10 + n), c.entry(b, 10 + i)) for b in (0, 7) for i, n in enumerate(good[:3])]
    c.check(done)
    err.zero_()
    lengths = [-3, 97] + [0] * 6
    accepted = [0] * 8
    new = api.compact(c.prob, c.caches, i32(lengths), i32([[0] + [-1] * 5] * 8), i32(accepted), **args)
    assert int(err) == api.DEVERR_LENGTH
    assert new.tolist() == [0, 96] + [1] * 6
    c.check(done)


@gpu
def test_many_rows_layers_streams_and_graphs(api):
    B, T = 66000, 2  # more rows than a grid's second dimension
    c = Case(api, layout="contiguous", kv="e4m3", heads=1, D=64, width=3, B=B, layers=1, seed=7)
    rng = np.random.default_rng(7)
    lengths = rng.integers(0, 2, B)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    new = api.compact(c.prob, c.caches, i32(lengths), i32(np.tile([0, 1], (B, 1))), i32(np.ones(B)), stream=s)
    s.synchronize()
    assert np.array_equal(new.cpu().numpy(), lengths + 2)
    c.check([])
    c = Case(api, layers=65, B=3, width=4, heads=1, D=64, page=8, seed=8)
    lengths, nodes, accepted = i32([3, 9, 0]), i32([[0, 2, 3, -1], [0, 2, -1, -1], [0, -1, -1, -1]]), i32([2, 1, 0])
    new, table = torch.zeros_like(lengths), c.table.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.compact(c.prob, c.caches, lengths, nodes, accepted, table=table, new_lengths=new)
    c.check([])
    lengths.copy_(i32([5, 9, 1]))
    graph.replay()
    assert new.tolist() == [8, 11, 2]
    c.check([(c.entry(0, 7), c.entry(0, 6)), (c.entry(0, 8), c.entry(0, 7)), (c.entry(1, 11), c.entry(1, 10))])


# ------------------------------------------------------------------ refusals (CPU)

def problem(api, **kw):
    args = dict(batch=2, num_q_heads=4, num_kv_heads=2, head_dim_qk=64, layout="paged", scale=0.1, page_size=4, width=3,
                num_blocks=6)
    args.update(kw)
    return api.problem(**args)


def test_argument_rules(api):
    L, inv, uns = api.lib(), api.ERR_INVALID_ARG, api.ERR_UNSUPPORTED
    ptrs = (ctypes.c_void_p * 2)(1 << 20, 1 << 24)
    odd = (ctypes.c_void_p * 2)(1 << 20, (1 << 24) + 4)
    null = (ctypes.c_void_p * 2)(1 << 20, 0)

    def caches(k=ptrs, v=ptrs, n=2):
        return api.DaCaches(n, ctypes.addressof(k) if k else None, ctypes.addressof(v) if v else None)

    def pages(p=None, c=None, src=1 << 12, dst=1 << 13, n=1, err=None):
        p, c = p or problem(api), c or caches()
        return L.decode_attn_copy_pages(ctypes.addressof(p), ctypes.addressof(c), src, dst, n, err, None)

    for kw in (dict(src=None), dict(dst=None), dict(src=2), dict(err=3), dict(n=-1), dict(c=caches(k=odd)),
               dict(c=caches(v=null)), dict(c=caches(v=None)), dict(c=caches(k=None)), dict(c=caches(n=0)),
               dict(p=problem(api, layout="contiguous")), dict(p=problem(api, page_size=0))):
        assert pages(**kw) == inv, kw
    assert pages(p=problem(api, head_dim_qk=96)) == uns
    assert L.decode_attn_copy_pages(ctypes.addressof(problem(api)), None, 4, 4, 1, None, None) == inv
    assert pages(n=0) == api.OK

    def compact(p=None, c=None, table=1 << 12, lengths=1 << 13, nodes=1 << 14, T=4, accepted=1 << 15, new=1 << 16, err=None):
        p, c = p or problem(api), c or caches()
        return L.decode_attn_compact(ctypes.addressof(p), ctypes.addressof(c), table, lengths, nodes, T, accepted, new, err, None)

    for kw in (dict(table=None), dict(lengths=None), dict(nodes=None), dict(accepted=None), dict(T=0), dict(T=65),
               dict(new=(1 << 16) + 2), dict(err=1), dict(new=1 << 13), dict(new=(1 << 14) + 28), dict(new=(1 << 15) - 4),
               dict(new=(1 << 12) + 20), dict(p=problem(api, layout="contiguous"))):
        assert compact(**kw) == inv, kw
    assert compact(p=problem(api, head_dim_qk=96)) == uns
    assert compact(p=problem(api, batch=0)) == api.OK


def test_python_checks(api):
    p = problem(api)
    k = [torch.zeros((6, 4, 2, 64), dtype=torch.bfloat16) for _ in range(4)]
    with pytest.raises(ValueError, match="overlap"):
        api.Caches(p, [k[0], k[1]], [k[2], k[1]])
    with pytest.raises(ValueError, match="each layer"):
        api.Caches(p, k[:2], k[:1])
    with pytest.raises(ValueError, match="each layer"):
        api.Caches(p, k[:2])
    with pytest.raises(ValueError, match="no caches"):
        api.Caches(p, [], [])
    with pytest.raises(ValueError, match="k holds"):
        api.Caches(problem(api, num_blocks=7), k[:2], k[2:])
    c = api.Caches(p, k[:2], k[2:])
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="another problem"):
        api.copy_pages(problem(api, num_blocks=7), c, one, one)
    with pytest.raises(ValueError, match="another problem"):
        api.copy_pages(problem(api, kv_dtype=api.KV_FP8_E4M3), c, one, one)
    with pytest.raises(ValueError, match="dst"):
        api.copy_pages(p, c, one, torch.zeros(2, dtype=torch.int32))
    two, nodes = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="table"):
        api.compact(p, c, two, nodes, two, new_lengths=two)
    with pytest.raises(ValueError, match="no CPU path"):
        api.compact(p, c, two, nodes, two.clone(), table=torch.zeros((2, 3), dtype=torch.int32), new_lengths=two.clone())
