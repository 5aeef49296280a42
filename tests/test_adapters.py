"""nvfp4_mm_adapters: each row's own low-rank adapter added to a shared matmul's
output, against the fp64 oracle, and the bitwise independence of a row from
the batch.

Tolerance.  Products are exact; every sum is fp32.  t adds 64 groups of 16
products per 1024-wide chunk and up to 8 chunks, the second product
3 * 128 / 16 = 24 groups; an fp32 accumulation step of the tensor core is off by
at most 2^-22 of the magnitudes it holds, so t and the product together stay
below (64 + 8 + 24 + 2) * 2^-22 < 2^-15 of mag = |scale| sum_r |B| sum_k |x| |A|.
The three bf16 terms hold t up to 2^-24 of it.  Adding to y rounds once more:
2^-24 of the result."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import step as OS

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from invariant_decode_attention_gb300 import api as _api
    _api.lib()
    return _api


class Case:
    def __init__(self, api, n, N, K, count, max_rank, *, x="bf16", ids=None, ranks="mixed", seed=0,
                 garbage=True):
        g = torch.Generator().manual_seed(seed)
        self.n, self.N, self.K = n, N, K
        self.x = torch.randn((n, K), generator=g).to(torch.bfloat16 if x == "bf16" else torch.float32)
        self.y = torch.randn((n, N), generator=g)
        self.a = (torch.randn((count, max_rank, K), generator=g) * K ** -0.5).to(torch.bfloat16)
        self.b = (torch.randn((count, N, max_rank), generator=g) * 0.1).to(torch.bfloat16)
        self.scales = torch.rand(count, generator=g) + 0.5
        self.ranks = None
        if ranks == "mixed":  # 0, 1, odd ones and the full rank among them
            self.ranks = torch.randint(0, max_rank + 1, (count,), generator=g, dtype=torch.int32)
            self.ranks[0] = max_rank
            if count > 2:
                self.ranks[1], self.ranks[2] = 0, 1
        self.ids = (torch.randint(-1, count, (n,), generator=g, dtype=torch.int32) if ids is None
                    else torch.as_tensor(ids, dtype=torch.int32))
        a, b = self.a.clone(), self.b.clone()
        if garbage and self.ranks is not None:  # nothing past a rank may show
            for i, r in enumerate(self.ranks.tolist()):
                a[i, r:] = float("nan")
                b[i, :, r:] = float("inf")
        self.handle = api.Adapters(a.cuda(), b.cuda(),
                                   None if self.ranks is None else self.ranks.cuda(),
                                   self.scales.cuda())
        self.api = api

    def run(self, rows=None, **kw):
        rows = torch.arange(self.n) if rows is None else torch.as_tensor(rows, dtype=torch.int64)
        y = self.y[rows].cuda()
        out = torch.full_like(y, float("nan"))
        kw.setdefault("out", out)
        return self.api.nvfp4_adapters(self.x[rows].cuda(), self.handle, self.ids[rows].cuda(), y,
                                       **kw)

    def check(self, out, rows=None):
        rows = np.arange(self.n) if rows is None else np.asarray(rows)
        ref, mag = OS.adapters(self.x[rows].double().numpy(), self.y[rows].numpy(),
                               self.a.double().numpy(), self.b.double().numpy(),
                               self.ids[rows].numpy(),
                               None if self.ranks is None else self.ranks.numpy(),
                               self.scales.numpy())
        err = np.abs(out.double().cpu().numpy() - ref)
        tol = 2.0 ** -24 * np.abs(ref) + 2.0 ** -15 * mag + 1e-40
        assert np.all(err <= tol), float((err / tol).max())


@gpu
@pytest.mark.parametrize("n,N,K,count,max_rank,x", [
    (1, 128, 64, 1, 16, "bf16"), (1, 256, 4096, 3, 64, "fp32"), (7, 128, 576, 4, 48, "bf16"),
    (32, 384, 1088, 2, 128, "fp32"), (33, 128, 512, 40, 16, "bf16"), (100, 256, 1536, 5, 112, "bf16"),
    (300, 640, 640, 7, 32, "fp32"), (65, 128, 8192, 6, 64, "bf16"),
])
def test_against_oracle(api, n, N, K, count, max_rank, x):
    c = Case(api, n, N, K, count, max_rank, x=x, seed=n + K)
    both = torch.full((n, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = api.adapters_workspace(n, N, K, c.handle)
    out = c.run(out_bf16=both, ws=ws)
    c.check(out)
    assert torch.equal(both, out.to(torch.bfloat16))
    assert api.nvfp4_read_error(ws) == 0


@gpu
def test_prompts_in_runs(api):
    # runs of rows that cross tiles, a run of one, rows without an adapter
    ids = [0] * 140 + [3] * 33 + [-1] * 5 + [1] + [2] * 64 + [-1] * 40 + [0] * 3
    c = Case(api, len(ids), 256, 1024, 4, 64, ids=ids, ranks=None, seed=4)
    c.check(c.run())


@gpu
def test_many_windows(api):
    # rows are grouped 512 at a time; sampled rows against the oracle, and bit for
    # bit the same as those rows in a small call
    n = 4130
    ids = np.sort(np.arange(n) % 5) - 1
    c = Case(api, n, 128, 2112, 4, 48, ids=ids, seed=6)
    out = c.run()
    rows = [0, 31, 32, 900, 1652, 2477, 2478, 3303, 4129]
    c.check(out[rows], rows)
    assert torch.equal(c.run(rows), out[rows])


@gpu
def test_row_bits_do_not_depend_on_the_batch(api):
    c = Case(api, 200, 256, 1600, 9, 64, seed=12)
    full = c.run()
    g = torch.Generator().manual_seed(3)
    for n in (1, 2, 8, 31, 33, 64, 150):
        rows = torch.randperm(200, generator=g)[:n]
        assert torch.equal(c.run(rows), full[rows]), n
    # all rows on one adapter, alone and together, at every place of a tile
    d = Case(api, 80, 128, 640, 2, 32, ids=[1] * 80, ranks=None, seed=13)
    full = d.run()
    for i in (0, 7, 8, 15, 16, 31, 32, 63, 64, 79):
        assert torch.equal(d.run([i])[0], full[i])
    assert torch.equal(d.run(list(range(79, -1, -1))), full.flip(0))


@gpu
def test_in_place_and_rows_without_an_adapter(api):
    c = Case(api, 50, 256, 512, 3, 32, seed=21)
    apart = c.run()
    none = c.ids < 0
    assert none.any() and torch.equal(apart[none].cpu(), c.y[none])
    y = c.y.cuda()
    both = torch.full((50, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = api.nvfp4_adapters(c.x.cuda(), c.handle, c.ids.cuda(), y, out_bf16=both)
    assert out is y and torch.equal(y, apart) and torch.equal(both, apart.to(torch.bfloat16))


@gpu
def test_bad_values_stay_in_their_row(api):
    ids = [0, 1, 2, 0, 1, 2, -1, 0]
    c = Case(api, 8, 128, 256, 3, 16, ids=ids, ranks=None, seed=8)
    clean = c.run()
    nan, inf = float("nan"), float("inf")
    c.x[3, 7], c.y[4, 5] = nan, inf
    c.handle.b[2, 9, 3] = inf  # all rows of adapter 2, output 9
    out = c.run()
    assert torch.isnan(out[3]).all()
    assert out[4, 5] == inf
    assert not torch.isfinite(out[[2, 5], 9]).any()
    keep = torch.ones_like(clean, dtype=torch.bool)
    keep[3], keep[4, 5], keep[2, 9], keep[5, 9] = False, False, False, False
    assert torch.equal(out[keep], clean[keep])


@gpu
def test_an_infinite_low_rank_value_stays_infinite(api):
    # t overflows to +inf: B's signs decide, no NaN from splitting t
    x = torch.full((1, 64), 3e38, dtype=torch.bfloat16, device="cuda")
    a = torch.ones((1, 16, 64), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros((1, 128, 16), dtype=torch.bfloat16, device="cuda")
    b[0, :64] = 1
    b[0, 64:] = -1
    y = torch.zeros((1, 128), device="cuda")
    out = api.nvfp4_adapters(x, api.Adapters(a, b), torch.zeros(1, dtype=torch.int32, device="cuda"), y)
    assert torch.all(out[0, :64] == float("inf")) and torch.all(out[0, 64:] == -float("inf"))


@gpu
def test_an_infinite_weight_gives_what_the_formula_gives(api):
    # t = 1.5 (its lower bf16 terms are zero) against an infinite B: an infinity of the
    # product's sign; NaN only where t is zero or infinities of both signs meet
    nan, inf = float("nan"), float("inf")
    x = torch.zeros((3, 64), dtype=torch.bfloat16)
    x[:, 0] = torch.tensor([1.5, -1.5, 0.0])
    a = torch.zeros((1, 16, 64), dtype=torch.bfloat16)
    a[0, :, 0] = 1
    b = torch.ones((1, 128, 16), dtype=torch.bfloat16)
    b[0, 3, 2], b[0, 4, 2], b[0, 5, 7], b[0, 5, 8], b[0, 6, 1] = inf, -inf, inf, -inf, nan
    y = torch.full((3, 128), 0.25)
    y[1, 7] = inf
    out = api.nvfp4_adapters(x.cuda(), api.Adapters(a.cuda(), b.cuda()),
                             torch.zeros(3, dtype=torch.int32, device="cuda"), y.cuda()).cpu()
    want = torch.tensor([24.25, -23.75, 0.25])[:, None].repeat(1, 128)
    want[0, 3:5], want[1, 3:5] = torch.tensor([inf, -inf]), torch.tensor([-inf, inf])
    want[2, 3:5], want[:, 5:7], want[1, 7] = nan, nan, inf
    assert torch.equal(torch.nan_to_num(out, 7e7, 8e8, -8e8), torch.nan_to_num(want, 7e7, 8e8, -8e8))


@gpu
def test_a_low_rank_value_between_the_largest_of_bf16_and_fp32(api):
    # t = 2^127 (2 - 2^-7 + 1.5 * 2^-8): beyond bf16, a number in fp32
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    x[0, :2] = torch.tensor([torch.finfo(torch.bfloat16).max, 1.5 * 2.0 ** 119])
    x[1, :2] = -x[0, :2]
    a = torch.zeros((1, 16, 64), dtype=torch.bfloat16)
    a[0, 5, :2] = 1
    b = torch.zeros((1, 128, 16), dtype=torch.bfloat16)
    b[0, :64, 5], b[0, 64:, 5] = 0.5, -0.25
    y = torch.zeros((2, 128))
    out = api.nvfp4_adapters(x.cuda(), api.Adapters(a.cuda(), b.cuda()),
                             torch.zeros(2, dtype=torch.int32, device="cuda"), y.cuda()).cpu()
    t = 2.0 ** 127 * (2 - 2.0 ** -7 + 1.5 * 2.0 ** -8)
    assert torch.all(out[0, :64] == 0.5 * t) and torch.all(out[0, 64:] == -0.25 * t)
    assert torch.equal(out[1], -out[0])


@gpu
@pytest.mark.parametrize("max_rank", [48, 112])
def test_infinities_in_a_large_batch(api, max_rank):
    # rows with infinite x and infinite weights of some adapters among others: the kinds
    # of results are the formula's, all finite ones have the bits of a call without them
    inf, n, N = float("inf"), 700, 256
    c = Case(api, n, N, 2112, 4, max_rank, seed=71, garbage=False)
    c.ranks = torch.tensor([max_rank, 1, 2, 17], dtype=torch.int32)
    c.handle.ranks.copy_(c.ranks)
    clean = c.run()
    c.x[::9, 1500] = inf
    c.x[4::27, 3] = -inf
    c.b[1, 7, 0], c.b[1, 8, 0], c.b[3, 100, 16], c.b[0, 255, 5] = inf, -inf, inf, float("nan")
    c.handle.b.copy_(c.b)
    out = c.run().cpu()
    hit = torch.zeros((n, N), dtype=torch.bool)
    for i in range(n):
        d = int(c.ids[i])
        if d < 0:
            continue
        r = int(c.ranks[d])
        t = c.a[d, :r].double() @ c.x[i].double()
        want = c.y[i].double() + float(c.scales[d]) * (c.b[d, :, :r].double() * t).sum(1)
        odd = ~torch.isfinite(want)
        assert torch.equal(torch.isnan(out[i]), torch.isnan(want)), i
        assert torch.equal(out[i][torch.isinf(want)].double(), want[torch.isinf(want)]), i
        hit[i] = odd
    assert torch.isinf(out[hit]).sum() > 1000 and torch.isnan(out[hit]).sum() > 1000
    assert torch.equal(out[~hit], clean.cpu()[~hit])


@gpu
@pytest.mark.parametrize("max_rank,K", [(16, 64), (64, 64), (64, 2176), (128, 2176)])
def test_low_rank_values_keep_all_their_bits(api, max_rank, K):
    """One-hot rows, so that out = fp32(scale * x) exactly: 24 bits need all three terms.
    Every rank meets every place of a tile."""
    g = torch.Generator().manual_seed(max_rank + K)
    col = torch.arange(max_rank) * (K // max_rank)  # the column that rank r picks
    a = torch.zeros((2, max_rank, K))
    a[:, torch.arange(max_rank), col] = 1
    N = 256
    b = (torch.arange(N)[:, None] % max_rank == torch.arange(max_rank)).float().repeat(2, 1, 1)
    scales = torch.tensor([1.9999998807907104, -1.4142135381698608])
    handle = api.Adapters(a.to(torch.bfloat16).cuda(), b.to(torch.bfloat16).cuda(), None, scales.cuda())
    rank = (torch.arange(64)[:, None] + torch.arange(0, max_rank, 16)).T.reshape(-1) % max_rank
    rank = torch.cat([(rank + s) % max_rank for s in range(16)])
    n = len(rank)
    ids = (torch.arange(n) // 512 % 2).int()  # full tiles, whole windows of one adapter
    x = torch.zeros((n, K))
    value = torch.randn(n, generator=g).to(torch.bfloat16).float()
    x[torch.arange(n), col[rank]] = value
    out = api.nvfp4_adapters(x.cuda(), handle, ids.cuda(), torch.zeros((n, N), device="cuda"))
    product = scales[ids.long()] * value
    want = torch.where(torch.arange(N) % max_rank == rank[:, None], product[:, None], 0.0)
    assert torch.equal(out.cpu(), want)
    assert (product != product.to(torch.bfloat16).float()).float().mean() > 0.9


@gpu
@pytest.mark.parametrize("max_rank,x,K", [(64, "bf16", 1088), (64, "fp32", 1088), (128, "bf16", 1088),
                                          (128, "fp32", 1088), (64, "fp32", 2112), (128, "bf16", 2112)])
def test_many_full_tiles_for_each_cta(api, max_rank, x, K):
    """More units than the CTAs have stages, slots and accumulators, at full tiles: 152
    CTAs take eight units of 128 features, or eight of a tile and a part of K, from
    four tiles.  Every element against fp64, and some rows bit for bit alone."""
    n, N, count = 40000, 256, 5
    ids = np.arange(n) * count // n
    c = Case(api, n, N, K, count, max_rank, x=x, ids=ids, ranks=None, seed=max_rank)
    both = torch.empty((n, N), dtype=torch.bfloat16, device="cuda")
    out = c.run(out_bf16=both)
    assert torch.equal(both, out.to(torch.bfloat16))
    worst = 0.0
    for d in range(count):
        rows = torch.as_tensor(ids == d)
        xr = c.x[rows].cuda().to(torch.bfloat16).double()
        a, b, s = c.a[d].cuda().double(), c.b[d].cuda().double(), float(c.scales[d])
        ref = c.y[rows].cuda().double() + s * (xr @ a.T) @ b.T
        mag = s * (xr.abs() @ a.abs().T) @ b.abs().T
        err = (out[rows.cuda()].double() - ref).abs()
        worst = max(worst, float((err / (2.0 ** -24 * ref.abs() + 2.0 ** -15 * mag)).max()))
    assert worst <= 1, worst
    rows = [0, 63, 64, 511, 512, 7999, 8000, 20011, 39999]
    assert torch.equal(c.run(rows), out[rows])


@gpu
def test_error_bits(api):
    c = Case(api, 40, 128, 256, 3, 16, ranks=None, seed=5)
    ws = api.adapters_workspace(40, 128, 256, c.handle)
    c.ids[35] = 3
    c.ids[36] = 2 ** 31 - 1
    out = c.run(ws=ws)
    assert api.nvfp4_read_error(ws) == api.DEVERR_INDEX
    assert torch.equal(out[35:37].cpu(), c.y[35:37])  # as without an adapter
    c.ids[35:37] = -1
    c.check(out)
    # ranks are clamped; the next call clears the word
    c.handle = api.Adapters(c.handle.a, c.handle.b, torch.tensor([17, 5, -1], dtype=torch.int32,
                                                                 device="cuda"), c.scales.cuda())
    c.ranks = torch.tensor([16, 5, 0])
    c.check(c.run(ws=ws))
    assert api.nvfp4_read_error(ws) == api.DEVERR_LENGTH
    c.ids[:] = 1
    c.run(ws=ws)
    assert api.nvfp4_read_error(ws) == 0


@gpu
def test_more_rows_than_a_slab(api):
    # two sets of launches, the second of one window: it keeps the first one's errors
    slab = 1 << 18
    n = slab + 300
    ids = np.full(n, -1)
    ids[[0, 700, 70000, slab - 1, slab, slab + 40, n - 1]] = [0, 1, 0, 1, 1, 0, 1]
    ids[5] = 2  # there is none
    c = Case(api, n, 128, 64, 2, 16, ids=ids, ranks=None, seed=31)
    ws = api.adapters_workspace(n, 128, 64, c.handle)
    out = c.run(ws=ws)
    assert api.nvfp4_read_error(ws) == api.DEVERR_INDEX
    rows = np.flatnonzero((ids == 0) | (ids == 1))
    c.check(out[torch.as_tensor(rows, device="cuda")], rows)
    assert torch.equal(c.run(rows), out[torch.as_tensor(rows, device="cuda")])
    others = torch.as_tensor((ids < 0) | (ids == 2))
    assert torch.equal(out.cpu()[others], c.y[others])


@gpu
def test_own_memory_on_another_stream(api):
    # workspaces made by the call belong to its stream: calls in a row on two
    # streams, without waiting for one another
    c = Case(api, 90, 256, 1088, 6, 64, seed=18)
    want = c.run()
    x, ids, y = c.x.cuda(), c.ids.cuda(), c.y.cuda()
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(y) for _ in range(12)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        api.nvfp4_adapters(x, c.handle, ids, y, out=out, stream=sides[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)


@gpu
def test_repeats_stream_and_graph(api):
    c = Case(api, 90, 384, 1088, 6, 64, seed=17)
    ws = api.adapters_workspace(90, 384, 1088, c.handle)
    ws.fill_(255)  # no initialisation needed
    first = c.run(ws=ws).clone()
    for _ in range(6):
        assert torch.equal(c.run(ws=ws), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x, ids, y = c.x.cuda(), c.ids.cuda(), c.y.cuda()
    out = torch.zeros_like(y)
    torch.cuda.synchronize()
    api.nvfp4_adapters(x, c.handle, ids, y, out=out, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.nvfp4_adapters(x, c.handle, ids, y, out=out, ws=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    # other rows through the same graph
    ids.copy_(ids.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    c.ids = c.ids.flip(0)
    c.check(out)


@gpu
@pytest.mark.parametrize("n", [1, 20, 90])
def test_replays_see_what_changed_between_them(api, n):
    # parts of the second kernel start before the first one has ended: everything
    # they read is what was there when the call began
    c = Case(api, n, 1024, 1088, 6, 64, seed=n, garbage=False)
    ws = api.adapters_workspace(n, 1024, 1088, c.handle)
    x, ids, y = c.x.cuda(), c.ids.cuda(), c.y.cuda()
    both = torch.empty((n, 1024), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):  # in place: each call reads what the last one wrote
            api.nvfp4_adapters(x, c.handle, ids, y, out_bf16=both, ws=ws)
    g = torch.Generator().manual_seed(n)
    for _ in range(6):
        c.ids = torch.randint(-1, 6, (n,), generator=g, dtype=torch.int32)
        c.ranks = torch.randint(0, 65, (6,), generator=g, dtype=torch.int32)
        c.scales = torch.rand(6, generator=g) + 0.5
        c.y = torch.randn((n, 1024), generator=g)
        ids.copy_(c.ids), y.copy_(c.y), c.handle.ranks.copy_(c.ranks), c.handle.scales.copy_(c.scales)
        graph.replay()
        torch.cuda.synchronize()
        for _ in range(3):
            c.y = c.run(ws=ws).cpu()
            torch.cuda.synchronize()
        assert torch.equal(y.cpu(), c.y) and torch.equal(both.cpu(), c.y.to(torch.bfloat16))


@gpu
def test_no_rows(api):
    c = Case(api, 3, 128, 64, 2, 16)
    assert c.run([]).shape == (0, 128)


@gpu
def test_a_call_without_rows_has_no_errors(api):
    # its workspace needs no initialisation either, and an earlier call's bits go
    c = Case(api, 3, 128, 64, 2, 16, ranks=None)
    ws = api.adapters_workspace(3, 128, 64, c.handle)
    ws.fill_(255)
    c.run([], ws=ws)
    assert api.nvfp4_read_error(ws) == 0
    c.ids[1] = 2
    c.run(ws=ws)
    c.run([], ws=ws)
    assert api.nvfp4_read_error(ws) == 0


# ------------------------------------------------------------------ refusals (no GPU)

def test_argument_rules(api):
    L, vp = api.lib(), ctypes.c_void_p
    fake = 1 << 20  # never dereferenced: every case fails before any device work
    size = L.nvfp4_mm_adapters_workspace_bytes
    # header, tiles per window, the tiles' ids, sizes and places, the rows in their
    # order, t per 1024 of K
    assert size(4, 128, 1088, 3, 64) == 6 * 256 + 2 * 4 * 64 * 4
    assert size(1 << 19, 128, 64, 1, 16) == size(1 << 18, 128, 64, 1, 16)  # rows in slabs
    for shape in ((-1, 128, 64, 1, 16), (1, 100, 64, 1, 16), (1, 128, 96, 1, 16), (1, 128, 64, 0, 16),
                  (1, 128, 64, 1, 8), (1, 128, 64, 1, 144), (1, 128, 64, 1, 24), (1 << 20, 128, 2048, 1, 16),
                  (1, 128, api.ADAPTER_MAX_K + 64, 1, 16)):
        assert size(*shape) == 0, shape

    def call(x=fake, xd=0, n=4, N=128, K=64, a=fake, b=fake, count=2, rank=16, ranks=fake, scales=fake,
             ids=fake, y=1 << 24, out=1 << 28, ob=1 << 30, ws=fake, wsb=1 << 30):
        p = lambda v: None if v is None else vp(v)  # noqa: E731
        return L.nvfp4_mm_adapters(p(x), xd, n, N, K, p(a), p(b), count, rank, p(ranks), p(scales),
                                   p(ids), p(y), p(out), p(ob), p(ws), wsb, None)
    bad = api.ERR_INVALID_ARG
    assert call(xd=2) == bad
    assert call(N=64) == api.ERR_UNSUPPORTED and call(rank=20) == api.ERR_UNSUPPORTED
    assert call(n=0, x=None, a=None, b=None, ids=None, y=None, out=None, ws=None) == api.OK
    for name in ("x", "a", "b", "ids", "y", "out"):
        assert call(**{name: None}) == bad, name
    for name in ("x", "a", "b", "y", "out"):
        assert call(**{name: (1 << 26) + 8}) == bad, name
    for name in ("ids", "ranks", "scales"):
        assert call(**{name: fake + 2}) == bad, name
    assert call(ob=fake + 8) == bad
    assert call(out=(1 << 24) + 512) == bad  # overlaps y
    assert call(out=fake) == bad and call(ob=fake) == bad                       # over x
    assert call(ob=1 << 24) == bad and call(ob=(1 << 28) + 1024) == bad         # over y, over out
    assert call(xd=1, ob=fake + 512, wsb=0) == api.ERR_WORKSPACE                # just behind x
    assert call(ws=None) == api.ERR_WORKSPACE
    assert call(ws=fake + 16) == api.ERR_WORKSPACE
    assert call(wsb=100) == api.ERR_WORKSPACE


def test_python_refusals(api):
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    f32, i32 = torch.float32, torch.int32
    with pytest.raises(ValueError, match="must be"):
        api.Adapters(t(2, 16, 64), t(3, 128, 16))
    with pytest.raises(ValueError, match="must be"):
        api.Adapters(t(2, 16, 64), t(2, 128, 32))
    with pytest.raises(ValueError, match="ranks"):
        api.Adapters(t(2, 16, 64), t(2, 128, 16), t(3, dtype=i32))
    with pytest.raises(ValueError, match="scales"):
        api.Adapters(t(2, 16, 64), t(2, 128, 16), None, t(2))
    with pytest.raises(ValueError, match="a must be"):
        api.Adapters(t(2, 16, 64, dtype=f32), t(2, 128, 16))
    h = api.Adapters(t(2, 16, 64), t(2, 128, 16))
    ok = dict(x=t(3, 64), ids=t(3, dtype=i32), y=t(3, 128, dtype=f32))

    def refused(match, **kw):
        a = {**ok, **kw}
        with pytest.raises(ValueError, match=match):
            api.nvfp4_adapters(a.pop("x"), h, a.pop("ids"), a.pop("y"), **a)
    refused("CUDA device")
    refused("float32 or bfloat16", x=t(3, 64, dtype=torch.float16))
    refused("columns", x=t(3, 128))
    refused("contiguous", x=t(3, 128)[:, ::2])
    refused("ids", ids=t(2, dtype=i32))
    refused("ids", ids=t(3, dtype=torch.int64))
    refused("y must", y=t(3, 128))
    refused("out must", out=t(3, 64, dtype=f32))
    refused("out_bf16", out_bf16=t(3, 128, dtype=f32))
    refused("ws", ws=t(4096, dtype=f32))
    big = api.Adapters(t(1, 24, 64), t(1, 128, 24))
    with pytest.raises(api.DecodeAttnError):
        api.adapters_workspace(1, 128, 64, big)


def test_oracle_on_a_hand_made_case():
    a = np.array([[[1.0, 2.0], [0.0, 1.0]]])
    b = np.array([[[1.0, 0.0], [2.0, -1.0]]])
    out, mag = OS.adapters([[1.0, -1.0], [1.0, 1.0]], [[10.0, 20.0], [1.0, 2.0]], a, b, [0, -1],
                           scales=[0.5])
    # t = (-1, -1); B t = (-1, -1); halved
    assert out.tolist() == [[9.5, 19.5], [1.0, 2.0]]
    assert mag.tolist() == [[1.5, 3.5], [0.0, 0.0]]
    out, _ = OS.adapters([[1.0, -1.0]], [[0.0, 0.0]], a, b, [0], ranks=[1])
    assert out.tolist() == [[-1.0, -2.0]]
