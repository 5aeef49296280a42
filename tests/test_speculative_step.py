"""One step over drafted tokens as a server makes it: the trees' tokens normed, rotated and
appended at entries of their own, attended to, verified, and the accepted entries moved
behind their contexts; then the caches are what a plain append of the accepted
tokens would have left, and plain decode attention reads them."""

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
KV = ("bf16", "e4m3", "nvfp4")
B, T, H_q, H, D, PAGE, WIDTH, LAYERS, V = 5, 7, 8, 2, 128, 16, 12, 2, 4001


@pytest.fixture(scope="module")
def api():
    from invariant_decode_attention_gb300 import api as _api
    _api.lib()
    return _api


class Server:
    def __init__(self, api, kv, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        self.kv = kv
        pages = B * WIDTH + 4
        self.table = torch.randperm(pages, generator=self.g)[:B * WIDTH].view(B, WIDTH).int().cuda()
        self.prob = api.problem(batch=B, num_q_heads=H_q, num_kv_heads=H, head_dim_qk=D, layout="paged", scale=D ** -0.5,
                                page_size=PAGE, width=WIDTH, num_blocks=pages, kv_dtype=KV.index(kv), k_scale=0.05,
                                v_scale=0.02)
        m = pages * PAGE * H * D
        size = {"bf16": 2 * m, "e4m3": m, "nvfp4": m // 2 + m // 16}[kv]
        self.bytes = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2 * LAYERS)]
        view = [t.view(torch.bfloat16) if kv == "bf16" else t for t in self.bytes]
        self.k, self.v = view[:LAYERS], view[LAYERS:]
        self.caches = api.Caches(self.prob, self.k, self.v)
        inv = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)).float().cuda()
        self.rope = api.rope(inv)
        w = [torch.randn(D, generator=self.g).abs().bfloat16().cuda() for _ in range(2)]
        self.norm = api.head_norm(*w, eps=1e-6)
        self.ws, self.vws = api.tree_workspace(self.prob, T), api.verify_workspace(B, T, V)
        self.pages = pages

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g)

    def i32(self, x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    def append(self, api, layer, qkv, positions, rows, entries=None):
        n = qkv.shape[0]
        q, k, v = (qkv[:, a:b].view(n, -1, D) for a, b in ((0, H_q * D), (H_q * D, (H_q + H) * D),
                                                          ((H_q + H) * D, (H_q + 2 * H) * D)))
        return api.append(self.prob, self.rope, k, v, self.k[layer], self.v[layer], positions, rows=rows,
                          table=self.table, q_new=q, norm=self.norm, entries=entries)

    def entry_bytes(self, layer, b, j):
        """The stored bytes of an entry, K and V."""
        at = int(self.table[b, j // PAGE]) * PAGE + j % PAGE
        got = []
        for t in (self.bytes[layer], self.bytes[LAYERS + layer]):
            m = self.pages * PAGE * H * D
            parts = [t] if self.kv != "nvfp4" else [t[:m // 2], t[m // 2:]]
            got += [p.view(self.pages * PAGE, -1)[at].cpu() for p in parts]
        return torch.cat(got)


def depths(par):
    d = []
    for p in par:
        d.append(0 if p < 0 else d[p] + 1)
    return d


@gpu
@pytest.mark.parametrize("kv", KV)
def test_a_step(api, kv):
    s = Server(api, kv)
    lengths = [40, 0, 17, 63, 100]
    # the contexts
    rows = np.repeat(np.arange(B), lengths)
    pos = np.concatenate([np.arange(n) for n in lengths])
    for layer in range(LAYERS):
        s.append(api, layer, s.rand(len(rows), (H_q + 2 * H) * D).cuda(), s.i32(pos), s.i32(rows))
    # the drafted trees
    par = np.array([[-1, 0, 0, 1, 1, 2, 5], [-1, 0, 1, 2, 3, 4, 5], [-1, 0, 0, 0, 3, 3, 4], [-1, 0, 1, 1, 2, 2, 3],
                    [-1, 0, 0, 1, 2, 3, 4]])
    dep = np.array([depths(p) for p in par])
    at = np.array(lengths)[:, None] + np.arange(T)
    tree_rows = s.i32(np.repeat(np.arange(B), T))
    positions = s.i32((np.array(lengths)[:, None] + dep).reshape(-1))
    qkv = [s.rand(B * T, (H_q + 2 * H) * D).cuda() for _ in range(LAYERS)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # what the target answers at the nodes, and tokens that it likes
    logits = (s.rand(B, T, V) * 2).cuda()
    tokens = torch.zeros((B, T), dtype=torch.int32)
    for b in range(B):
        for t in range(1, T):
            tokens[b, t] = int(logits[b, par[b, t]].float().topk(4).indices[t % 4])
    u, final = torch.rand((B, T), generator=s.g).cuda() * 0.05, torch.rand(B, generator=s.g).cuda()
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    outs = [torch.zeros((B, T, H_q, D), dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)]
    acc, nodes, toks = s.i32(np.zeros(B)), s.i32(np.zeros((B, T))), s.i32(np.zeros((B, T)))
    len_t, par_t, at_t, tok_t = s.i32(lengths), s.i32(par), s.i32(at.reshape(-1)), tokens.cuda()
    lse = torch.zeros((B, T, H_q), device="cuda")

    def step():
        for layer in range(LAYERS):
            q = s.append(api, layer, qkv[layer], positions, tree_rows, entries=at_t)
            api.tree(s.prob, q.view(B, T, H_q, D), s.k[layer], s.v[layer], len_t, parents=par_t, table=s.table,
                     out=outs[layer], lse=lse, ws=s.ws, err=err)
        api.nvfp4_verify(logits, tok_t, u, final, parents=par_t, accepted=acc, nodes=nodes, out=toks, ws=s.vws, err=err)
        api.compact(s.prob, s.caches, len_t, nodes, acc, table=s.table, new_lengths=new, err=err)

    before = [t.clone() for t in s.bytes]
    step()
    torch.cuda.synchronize()
    assert int(err) == 0
    once = [t.clone() for t in s.bytes], [o.clone() for o in outs], toks.clone(), new.clone()
    assert int(acc.max()) >= 1  # the tokens are likely ones

    # the same step captured and replayed
    for t, b in zip(s.bytes, before):
        t.copy_(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(once[0], s.bytes))
    assert all(torch.equal(a, b) for a, b in zip(once[1], outs)) and torch.equal(once[2], toks)

    # a plain server that appends the accepted tokens one after the other holds the same bytes
    n_acc, paths = acc.tolist(), nodes.tolist()
    p = Server(api, kv)
    p.table.copy_(s.table)
    for t, b in zip(p.bytes, before):
        t.copy_(b)
    for layer in range(LAYERS):
        pick = [b * T + paths[b][i] for b in range(B) for i in range(n_acc[b] + 1)]
        r = [b for b in range(B) for _ in range(n_acc[b] + 1)]
        place = [lengths[b] + i for b in range(B) for i in range(n_acc[b] + 1)]
        q = p.append(api, layer, qkv[layer][pick], p.i32(place), p.i32(r))
        for b, j in zip(r, place):
            assert torch.equal(p.entry_bytes(layer, b, j), s.entry_bytes(layer, b, j)), (layer, b, j)
        # and its decode attention agrees with the tree's at the last accepted node
        last = [sum(n_acc[:b + 1]) + b for b in range(B)]
        o, l = torch.empty((B, H_q, D), dtype=torch.bfloat16, device="cuda"), torch.empty((B, H_q), device="cuda")
        api.forward(p.prob, api.INVARIANT, q[last].contiguous(), p.k[layer], p.v[layer], p.table, new,
                    api.workspace(p.prob), o, l)
        got = torch.stack([outs[layer][b, paths[b][n_acc[b]]] for b in range(B)])
        assert float((got.float() - o.float()).abs().max()) <= 0.125  # two bf16 steps of the largest
    assert new.tolist() == [n + a + 1 for n, a in zip(lengths, n_acc)]


@gpu
def test_a_fork(api):
    """A row forked in two: full pages shared, the last one copied; both then go on."""
    s = Server(api, "bf16", seed=1)
    L = 40  # two full pages and a half
    s.append(api, 0, s.rand(L, (H_q + 2 * H) * D).cuda(), s.i32(np.arange(L)), s.i32(np.zeros(L)))
    free = [p for p in range(s.pages) if p not in s.table.flatten().tolist()][0]
    s.table[1] = s.table[0]
    s.table[1, 2] = free
    api.copy_pages(s.prob, s.caches, s.table[0, 2:3].clone(), s.table[1, 2:3].clone())
    qkv = s.rand(2, (H_q + 2 * H) * D).cuda()
    q = s.append(api, 0, qkv, s.i32([L, L]), s.i32([0, 1]))
    for j in range(L):
        assert torch.equal(s.entry_bytes(0, 0, j), s.entry_bytes(0, 1, j))
    assert not torch.equal(s.entry_bytes(0, 0, L), s.entry_bytes(0, 1, L))
    out, _ = api.tree(s.prob, torch.cat([q, q[:1], q[:1], q[:1]]).view(B, 1, H_q, D), s.k[0], s.v[0],
                      s.i32([L, L, 0, 0, 0]), table=s.table, counts=s.i32([1, 1, 0, 0, 0]))
    assert not torch.equal(out[0], out[1])
