"""nvfp4_mm_verify: which drafted tokens stand and the token after them, against the
definition in fp64.

All results are whole numbers and have to be equal.  A decision differs only if a random
number falls between a border here and there: borders of accepted tokens are off by an
fp32 sum's error (below 2^-20 of p), those of the next token by 2^-38 of a weight.  The
random numbers of these cases are fixed and lie further away than that: `decide` asserts a
distance of 1e-6 for acceptance and 1e-11 for the next token."""

import ctypes

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from invariant_decode_attention_gb300 import api as _api
    _api.lib()
    return _api


def probabilities(x, tau):
    x = np.where(np.isnan(x), -np.inf, x)
    m = x.max()
    if m == -np.inf:
        return np.zeros_like(x)
    if m == np.inf:
        w = (x == np.inf).astype(float)
    else:
        w = np.exp((x - m) / tau)
    return w / w.sum()


def decide(x, tokens, u, final, par, n, tau, draft=None):
    """(path of nodes, tokens) of one request; x: [T, V] fp64."""
    V = x.shape[1]
    path = [0]
    while True:
        i = path[-1]
        kids = [t for t in range(1, n) if par[t] == i and 0 <= tokens[t] < V]
        took = None
        if tau == 0:
            y = np.where(np.isnan(x[i]), -np.inf, x[i])
            best = int(y.argmax()) if y.max() > -np.inf else -1
            took = next((t for t in kids if tokens[t] == best), None)
        else:
            p, at, had = probabilities(x[i], tau), 0.0, set()
            for t in kids:
                if draft is not None:
                    q = draft[t, tokens[t]]
                    assert not (abs(u[i] * q - p[tokens[t]]) < 1e-6 * p[tokens[t]]), "too near a border"
                    yes = bool(u[i] * q < p[tokens[t]])
                else:
                    at += 0.0 if tokens[t] in had else p[tokens[t]]
                    had.add(tokens[t])
                    assert abs(u[i] - at) > 1e-6 or u[i] == 0, "too near a border"
                    yes = u[i] < at
                if yes:
                    took = t
                    break
        if took is None:
            break
        path.append(took)
    out = [int(tokens[t]) for t in path[1:]]
    if tau == 0:
        return path, out + [best]
    r = p.copy()
    if kids and draft is not None:
        q = draft[kids[0]].copy()
        q[~(q > 0)] = 0
        less = np.maximum(p - q, 0)
        r = less if less.sum() > 0 else p
    elif kids:
        r[[tokens[t] for t in kids]] = 0
        r = r if r.sum() > 0 else p
    total = np.cumsum(r)
    if total[-1] == 0:
        return path, out + [-1]
    limit = final * total[-1]
    v = int(np.searchsorted(total, limit, side="right"))
    near = np.abs(np.array([total[v], total[v - 1] if v else -1.0]) - limit).min()
    assert near > 1e-11 * total[-1] or final == 0, "too near a border"
    return path, out + [v]


class Case:
    def __init__(self, *, B=3, T=5, V=1000, x="fp32", tree=False, draft=False, taus=(1.0,), seed=0, spread=3.0,
                 counts=None, skew=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.B, self.T, self.V = B, T, V
        store = torch.randn((B, T, V + skew), generator=g) * spread
        self.x = (store.bfloat16() if x == "bf16" else store)[..., :V]  # rows that start anywhere
        self.par = np.tile(np.arange(-1, T - 1), (B, 1))
        if tree:
            self.par = np.stack([[-1] + [int(rng.integers(max(0, t - 4), t)) for t in range(1, T)] for _ in range(B)])
        self.tree = tree
        near = torch.stack([self.x[b, torch.tensor(self.par[b]).clamp(min=0)] for b in range(B)]).float()
        self.draft = torch.softmax(near + torch.randn((B, T, V), generator=g) * 0.5, -1)
        self.tokens = torch.multinomial(self.draft.view(B * T, V), 1, generator=g).view(B, T).int()
        self.use_draft = draft
        self.u, self.final = torch.rand((B, T), generator=g), torch.rand(B, generator=g)
        self.tau = torch.tensor([taus[b % len(taus)] for b in range(B)])
        self.counts = counts

    def run(self, api, **kw):
        c = lambda t: t.cuda()  # noqa: E731
        x = kw.pop("x", None)
        if x is None:
            x = torch.empty((self.B, self.T, self.x.stride(1)), dtype=self.x.dtype, device="cuda")[..., :self.V]
            x.copy_(self.x)
        kw.setdefault("parents", torch.tensor(self.par).int().cuda() if self.tree else None)
        kw.setdefault("draft", c(self.draft) if self.use_draft else None)
        kw.setdefault("counts", None if self.counts is None else torch.tensor(self.counts).int().cuda())
        return api.nvfp4_verify(x, c(self.tokens), c(self.u), c(self.final), temperature=c(self.tau), **kw)

    def check(self, got, rows=None):
        accepted, nodes, out = (t.cpu().numpy() for t in got)
        for b in range(self.B) if rows is None else rows:
            n = self.T if self.counts is None else max(0, min(self.T, self.counts[b]))
            path, toks = ([], []) if n == 0 else decide(
                self.x[b].double().numpy(), self.tokens[b].numpy(), self.u[b].double().numpy(), float(self.final[b]),
                self.par[b], n, float(self.tau[b]), self.draft[b].double().numpy() if self.use_draft else None)
            pad = [-1] * self.T
            assert accepted[b] == max(0, len(path) - 1), b
            assert nodes[b].tolist() == (path + pad)[:self.T], b
            assert out[b].tolist() == (toks + pad)[:self.T], b


GRID = [(x, tree, draft, T, V) for x in ("fp32", "bf16") for tree, draft in ((False, True), (False, False), (True, False))
        for T, V in ((1, 700), (5, 1), (4, 4099), (16, 20001), (8, 50000))]


@gpu
@pytest.mark.parametrize("x,tree,draft,T,V", GRID)
def test_against_definition(api, x, tree, draft, T, V):
    c = Case(B=11, T=T, V=V, x=x, tree=tree, draft=draft, taus=(1.0, 0.7, 0.0, 1.6), seed=T + V)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(c.run(api, err=err))
    assert int(err) == 0


@gpu
@pytest.mark.parametrize("draft", [False, True])
def test_large_vocabulary_and_wide_trees(api, draft):
    c = Case(B=3, T=64 if not draft else 33, V=131072, tree=not draft, draft=draft, seed=1)
    c.check(c.run(api))
    c = Case(B=1, T=2, V=1 << 19, draft=draft, x="bf16", seed=2)
    c.check(c.run(api))


@gpu
@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("skew", [1, 2, 3, 5])
def test_rows_that_start_anywhere(api, x, skew):
    c = Case(B=5, T=3, V=9001, x=x, draft=True, skew=skew, seed=skew)
    got = c.run(api)
    c.check(got)
    whole = c.x.contiguous()[:, :, :9001].cuda()
    again = c.run(api, x=whole)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@gpu
def test_ragged_counts(api):
    c = Case(B=6, T=7, V=3000, tree=True, counts=[7, 0, 1, 3, 9, -2], seed=4)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = c.run(api, err=err)
    assert int(err) == api.DEVERR_LENGTH
    c.check(got)


@gpu
def test_paths_of_every_length(api):
    # a draft that is the target: everything is accepted; one that never is: nothing
    c = Case(B=4, T=6, V=500, draft=True, seed=5)
    c.draft = torch.softmax(torch.cat([c.x[:, :1], c.x[:, :-1]], 1), -1)
    c.tokens = c.draft.argmax(-1).int()
    accepted, nodes, out = c.run(api)
    assert accepted.tolist() == [5] * 4 and nodes.tolist() == [list(range(6))] * 4
    assert torch.equal(out[:, :5].cpu(), c.tokens[:, 1:])
    c.check((accepted, nodes, out))
    for b in range(4):
        c.x[b, b, c.tokens[b, b + 1]] = -float("inf")  # node b + 1 cannot be accepted
    got = c.run(api)
    assert got[0].tolist() == [0, 1, 2, 3]
    c.check(got)


@gpu
@pytest.mark.parametrize("u", [0.0, 1.0 - 2.0 ** -24])
def test_the_ends_of_the_random_numbers(api, u):
    c = Case(B=4, T=4, V=3001, tree=True, seed=6)
    c.x[:, :, 2000:] = -float("inf")  # the last token that may come is 1999
    c.x[:, :, :7] = -float("inf")
    c.u[:], c.final[:] = u, u
    accepted, nodes, out = (t.cpu() for t in c.run(api))
    if u == 0:  # the first child with any probability, the lowest token that may come
        c.check((accepted, nodes, out))
    else:
        assert (accepted == 0).all()
        for b in range(4):
            kids = {int(c.tokens[b, t]) for t in range(1, 4) if c.par[b][t] == 0}
            assert int(out[b, 0]) == max(v for v in range(7, 2000) if v not in kids)


@gpu
def test_repeated_siblings_count_once(api):
    c = Case(B=1, T=5, V=10, tree=True, seed=7)
    c.par = np.array([[-1, 0, 0, 0, 0]])
    c.x[0, 0] = torch.log(torch.tensor([.1, .2, .3, .05, .05, .1, .05, .05, .05, .05]))
    c.tokens[0] = torch.tensor([0, 1, 1, 2, 1])
    for u, took in ((0.1, 1), (0.19, 1), (0.21, 3), (0.45, 3), (0.51, None), (0.9, None)):
        c.u[0, 0] = u
        got = c.run(api)
        assert got[1][0].tolist() == ([0, took] if took else [0, -1]) + [-1] * 3, u
        c.check(got)


@gpu
def test_what_is_left_when_everything_is_drafted(api):
    # two tokens, both drafted, share all of p; u just below 1 accepts one of them still
    c = Case(B=1, T=3, V=2, tree=True, seed=8)
    c.par = np.array([[-1, 0, 0]])
    c.tokens[0] = torch.tensor([0, 1, 0])
    c.u[0, 0] = 1 - 2.0 ** -24
    accepted, nodes, out = c.run(api)
    # (the border, 1, is 2^-24 away: within the fp32 sum's error of either side)
    assert nodes[0].tolist() in ([0, 2, -1], [0, -1, -1])
    assert int(accepted) == int(nodes[0, 1] == 2) and int(out[0, 0]) in (0, 1)
    # q = p where it matters: nothing is left of p - q, the target's own p takes over
    c = Case(B=1, T=2, V=3, draft=True, seed=9)
    c.draft[0, 1] = torch.tensor([1.0, 1.0, 1.0])
    c.u[0, 0], c.tokens[0, 1] = 0.999, 0
    c.x[0, 0] = torch.tensor([0.0, 0.5, 0.1])
    got = c.run(api)
    assert int(got[0]) == 0
    c.check(got)


@gpu
@pytest.mark.parametrize("x", ["fp32", "bf16"])
def test_special_logits(api, x):
    nan, inf = float("nan"), float("inf")
    c = Case(B=7, T=3, V=5000, x=x, seed=10, taus=(1.0, 0.0))
    c.x[0, :, ::2] = nan
    c.x[1, :, ::2] = nan
    c.x[2] = -inf
    c.x[3] = nan
    c.x[4, :, 1234] = inf
    c.x[4, :, 77] = inf
    c.x[5, :, 300] = inf
    c.x[6, 0] = 1.0  # all equal
    got = c.run(api)
    c.check(got)
    assert got[2][2, 0] == -1 and got[2][3, 0] == -1


@gpu
def test_greedy_ties_go_to_the_lowest(api):
    c = Case(B=2, T=4, V=40000, tree=True, taus=(0.0,), seed=11)
    c.par = np.array([[-1, 0, 0, 1]] * 2)
    c.x = torch.zeros_like(c.x)
    c.x[:, :, [123, 20000, 39999]] = 5.0
    c.tokens = torch.tensor([[0, 20000, 123, 123], [0, 123, 123, 123]]).int()
    got = c.run(api)
    assert got[1].tolist() == [[0, 2, -1, -1], [0, 1, 3, -1]]
    c.check(got)


@gpu
def test_temperatures_at_the_ends(api):
    c = Case(B=6, T=2, V=3000, taus=(1e-30, 1e30, -1.0, float("nan"), float("inf"), 1e-45), seed=12)
    got = c.run(api)
    for b, t in enumerate((0.0, None, 0.0, 0.0, None, 0.0)):
        best = int(c.x[b, 0].argmax())
        if t == 0.0:
            first = got[2][b, 0].item()
            assert first == best
        else:  # all tokens alike
            v = int(np.floor(float(c.final[b]) * 3000)) if got[0][b] == 0 else None
            assert v is None or abs(int(got[2][b, 0]) - v) <= 1


@gpu
def test_draft_values_that_are_none(api):
    c = Case(B=4, T=2, V=600, draft=True, seed=13)
    tok = [int(c.tokens[b, 1]) for b in range(4)]
    for b, q in enumerate((float("nan"), 0.0, float("inf"), -1.0)):
        c.draft[b, 1, tok[b]] = q
    got = c.run(api)
    assert got[0].tolist()[:3] == [0, 1, 0]  # refused, accepted, refused
    c.draft[3, 1] = float("nan")  # refused, and nothing is taken off p
    got = c.run(api)
    assert int(got[0][3]) == 0
    p = probabilities(c.x[3, 0].double().numpy(), 1.0)
    want = int(np.searchsorted(np.cumsum(p), float(c.final[3]) * 1.0, side="right"))
    assert int(got[2][3, 0]) == want


@gpu
@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [2, 40])
def test_negative_draft_values_refuse(api, x, T):
    """Whatever the target says of the token, and with nothing taken off p for it."""
    inf = float("inf")
    values = (-1.0, -1.0, -1.0, -inf, -1e-45, -3e38, -0.0)
    c = Case(B=7, T=T, V=900, x=x, draft=True, seed=17)
    last = T - 1  # the refusal is here, in either half of a warp's nodes
    c.u[:, :last - 1] = 0.0  # accepted up to there
    for b, q in enumerate(values):
        c.draft[b, last, int(c.tokens[b, last])] = q
    c.u[1, last - 1] = 0.0                             # 0 * q is -0
    c.x[2, last - 1, int(c.tokens[2, last])] = -inf    # no share of the target's, any q < 0 is less
    got = c.run(api)
    assert got[0].tolist() == [last - 1] * 6 + [last]  # (-0 is not negative)
    # the definition, which refuses at a NaN and takes nothing off p for it
    c.draft[c.draft < 0] = float("nan")
    c.check(got)


@gpu
def test_tokens_and_parents_out_of_range(api):
    c = Case(B=5, T=4, V=2000, tree=True, seed=14)
    c.u[:] = 1e-9  # the first child that can be accepted is
    c.par = np.array([[-1, 0, 0, 1]] * 5)
    c.tokens[0, 1], c.tokens[1, 1] = -1, 2000
    c.par[2][1], c.par[3][1], c.par[4][1] = 1, -2, -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = c.run(api, err=err)
    assert int(err) == api.DEVERR_INDEX
    assert got[1][:, :2].tolist() == [[0, 2]] * 5
    err.zero_()
    c.par[2:4, 1] = -1  # no error: not part of the tree
    c.tokens[:2, 1] = 5
    c.run(api, err=err)
    assert int(err) == 0


@gpu
def test_a_request_depends_on_itself_alone(api):
    c = Case(B=9, T=6, V=30001, draft=True, taus=(0.9,), seed=15)
    got = c.run(api)
    for b in (0, 4, 8):
        r = slice(b, b + 1)
        one = api.nvfp4_verify(c.x[r].cuda(), c.tokens[r].cuda(), c.u[r].cuda(), c.final[r].cuda(), draft=c.draft[r].cuda(),
                               temperature=c.tau[r].cuda())
        assert all(torch.equal(a[0], g[b]) for a, g in zip(one, got))


@gpu
def test_rows_beyond_32_bits(api):
    """Requests and nodes 2^32 and 2^30 elements apart, of logits and draft's probabilities."""
    c = Case(B=2, T=3, V=5003, x="bf16", draft=True, seed=23)
    want = c.run(api)
    c.check(want)
    apart = (1 << 32) + 6, (1 << 30) + 2
    size = apart[0] + 2 * apart[1] + 5003
    x = torch.empty(size, dtype=torch.bfloat16, device="cuda").as_strided((2, 3, 5003), (*apart, 1))
    draft = torch.empty(size, device="cuda").as_strided((2, 3, 5003), (*apart, 1))
    x.copy_(c.x)
    draft.copy_(c.draft)
    got = c.run(api, x=x, draft=draft)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    del x, draft
    torch.cuda.empty_cache()


@gpu
def test_tokens_are_distributed_as_the_targets(api):
    """Accepted or not, the first token has the target's distribution: 2^16 requests that
    differ in their random numbers alone, counts within six standard deviations."""
    B, V = 1 << 16, 6
    g = torch.Generator().manual_seed(16)
    p = torch.tensor([.05, .4, .15, .2, .12, .08])
    x = torch.log(p).expand(B, 4, V).contiguous().cuda()
    q = torch.tensor([.3, .1, .2, .1, .1, .2])
    draft = q.expand(B, 4, V).contiguous().cuda()
    tokens = torch.multinomial(q, B * 4, replacement=True, generator=g).view(B, 4).int().cuda()
    u, f = torch.rand((B, 4), generator=g).cuda(), torch.rand(B, generator=g).cuda()
    chain = api.nvfp4_verify(x, tokens, u, f, draft=draft)
    par = torch.tensor([-1, 0, 0, 1]).int().expand(B, 4).contiguous().cuda()
    fixed = torch.tensor([0, 3, 1, 3]).int().expand(B, 4).contiguous().cuda()
    tree = api.nvfp4_verify(x, fixed, u, f, parents=par)
    for got in (chain, tree):
        n = torch.bincount(got[2][:, 0].cpu(), minlength=V).double()
        assert ((n - B * p).abs() <= 6 * (B * p * (1 - p)).sqrt()).all(), n / B


@gpu
def test_streams_and_graphs(api):
    c = Case(B=6, T=5, V=12345, tree=True, seed=17)
    want = c.run(api)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.run(api, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    x, tokens, u, f = c.x.contiguous().cuda(), c.tokens.cuda(), c.u.cuda(), c.final.cuda()
    par, tau, ws = torch.tensor(c.par).int().cuda(), c.tau.cuda(), api.verify_workspace(6, 5, 12345)
    outs = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.nvfp4_verify(x, tokens, u, f, parents=par, temperature=tau, accepted=outs[0], nodes=outs[1], out=outs[2], ws=ws)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    g = torch.Generator().manual_seed(18)
    c.u, c.final = torch.rand((6, 5), generator=g), torch.rand(6, generator=g)
    u.copy_(c.u)
    f.copy_(c.final)
    graph.replay()
    c.check(outs)


# ------------------------------------------------------------------ refusals (CPU)

def packed(api, **kw):
    a = dict(B=2, T=4, V=100, xt=api.X_F32, x=1 << 20, xs=400, xn=100, draft=0, ds=0, dn=0, tokens=1 << 21, parents=0,
             counts=0, tau=0, u=1 << 22, f=1 << 23, accepted=1 << 24, nodes=1 << 25, out=1 << 26, err=0, ws=1 << 27,
             n=api.verify_workspace_bytes(2, 4, 100))
    a.update(kw)
    return api._VERIFY.pack(*a.values())


def test_argument_rules(api):
    L, inv, uns, wsp = api.lib(), api.ERR_INVALID_ARG, api.ERR_UNSUPPORTED, api.ERR_WORKSPACE
    call = lambda **kw: L.nvfp4_mm_verify(packed(api, **kw), None)  # noqa: E731
    assert L.nvfp4_mm_verify(None, None) == inv
    for kw in (dict(B=-1), dict(T=0), dict(V=0), dict(xt=5), dict(x=0), dict(tokens=0), dict(u=0), dict(f=0),
               dict(accepted=0), dict(nodes=0), dict(out=0), dict(x=(1 << 20) + 2), dict(tokens=(1 << 21) + 1),
               dict(xs=99), dict(xn=99), dict(xn=1 << 41), dict(draft=1 << 28, parents=1 << 12),
               dict(draft=1 << 28, ds=400, dn=99), dict(draft=1 << 28, ds=99, dn=100), dict(draft=(1 << 28) + 2, ds=400, dn=100),
               dict(err=2), dict(out=1 << 21), dict(nodes=(1 << 21) + 28), dict(accepted=1 << 22), dict(out=(1 << 25) + 4),
               dict(out=(1 << 20) + 400), dict(accepted=1 << 27), dict(draft=(1 << 24) - 8, ds=400, dn=100),
               dict(draft=(1 << 26) - 3000, ds=400, dn=100)):
        assert call(**kw) == inv, kw
    for kw in (dict(T=65), dict(V=(1 << 19) + 1)):
        assert call(**kw) == uns, kw
    for kw in (dict(ws=0), dict(ws=(1 << 27) + 8), dict(n=api.verify_workspace_bytes(2, 4, 100) - 1)):
        assert call(**kw) == wsp, kw
    assert call(B=0) == api.OK


def test_workspace_sizes(api):
    assert api.verify_workspace_bytes(2, 4, 100) >= 256
    assert api.verify_workspace_bytes(64, 8, 131072) >= 64 * 8 * 16 * 16
    for bad in ((-1, 4, 100), (2, 0, 100), (2, 65, 100), (2, 4, 0), (2, 4, (1 << 19) + 1)):
        assert api.verify_workspace_bytes(*bad) == 0
    with pytest.raises(api.DecodeAttnError):
        api.verify_workspace(2, 65, 100, device="cpu")


def test_python_checks(api):
    x, i, f = torch.zeros((2, 3, 50)), torch.zeros((2, 3), dtype=torch.int32), torch.zeros((2, 3))
    ws, row = torch.zeros(4096, dtype=torch.uint8), torch.zeros(2)
    ok = dict(ws=ws, accepted=row.int(), nodes=i.clone(), out=i.clone())
    with pytest.raises(ValueError, match="no CPU path"):
        api.nvfp4_verify(x, i, f, row, **ok)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        api.nvfp4_verify(x.double(), i, f, row, **ok)
    for kw, word in ((dict(draft=x.bfloat16()), "draft"), (dict(parents=i[:1]), "parents"), (dict(counts=row), "counts"),
                     (dict(temperature=row.double()), "temperature"), (dict(out=i[:, :2]), "out")):
        with pytest.raises(ValueError, match=word):
            api.nvfp4_verify(x, i, f, row, **{**ok, **kw})
    with pytest.raises(ValueError, match="strides"):
        api.nvfp4_verify(torch.zeros((2, 50, 3)).transpose(1, 2), i, f, row, **ok)


def test_the_definition_used_here():
    # hand-worked: p = (1/2, 1/4, 1/4); tokens 1 and 2 drafted as siblings
    x = np.log(np.array([[.5, .25, .25]] * 3))
    par, tok = [-1, 0, 0], [0, 1, 2]
    assert decide(x, tok, [.2, .9, .9], .3, par, 3, 1.0) == ([0, 1], [1, 0])
    assert decide(x, tok, [.4, .9, .9], .6, par, 3, 1.0) == ([0, 2], [2, 1])
    assert decide(x, tok, [.6, .9, .9], .9, par, 3, 1.0) == ([0], [0])  # only token 0 is left
    q = np.array([[0, 0, 0], [.25, .5, .25], [0, 0, 1.0]])
    chain = [-1, 0, 1]
    assert decide(x, [0, 1, 2], [.4, .2, .9], .1, chain, 3, 1.0, q) == ([0, 1, 2], [1, 2, 0])
    assert decide(x, [0, 1, 2], [.6, .2, .9], .9, chain, 3, 1.0, q) == ([0], [0])  # p - q is left at token 0 alone
