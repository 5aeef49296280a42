"""decode_attn_append_norm: heads normed, rotated and stored, drafted tokens at entries
of their own, against fp64.

Tolerance.  A normed value x r (w + add) carries the errors of a 128-term fp32 sum of
squares (at most 2^-20 of it, half of that in its root), a correctly rounded root, two
products and a sum: below 2^-19 of its magnitude.  The rotation adds 2^-20 (|a| + |b|)
as in plain appends.  Storing rounds once: 2^-8 of the value for bf16, 2^-4 for E4M3 (and
2^-10 of the scale where it has no smaller step), half the spacing of E2M1 for NVFP4."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8 as OF
from oracle import nvfp4 as ON
from oracle import step as OS

gpu = pytest.mark.gpu
KV = ("bf16", "e4m3", "nvfp4")
K_SCALE, V_SCALE = 1.0 / 48, 1.0 / 64


@pytest.fixture(scope="module")
def api():
    from invariant_decode_attention_gb300 import api as _api
    _api.lib()
    return _api


class Case:
    def __init__(self, api, *, n=20, layout="paged", kv="bf16", heads=(8, 2, 128), rope=(128, 0, False), x="bf16",
                 page=16, w="bf16", w_add=0.0, eps=1e-6, entries=True, which="qk", seed=0, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        H_q, H, D = heads
        self.kv, self.heads, self.n, self.eps, self.w_add = kv, heads, n, eps, w_add
        dt = torch.bfloat16 if x == "bf16" else torch.float32
        row = (torch.randn((n, (H_q + 2 * H) * D), generator=g) * torch.rand((n, 1), generator=g) * gain).to(dt).cuda()
        self.q = row[:, :H_q * D].view(n, H_q, D)
        self.k_new = row[:, H_q * D:(H_q + H) * D].view(n, H, D)
        self.v_new = row[:, (H_q + H) * D:].view(n, H, D)
        B, room = 4, 8 * page
        pick = torch.randperm(B * room, generator=g)[:n]
        rows, self.at = pick // room, pick % room
        self.pos = torch.randint(0, 5000, (n,), generator=g) if entries or layout == "indexed" else self.at
        self.table, width = None, room
        if layout == "paged":
            width, blocks = 8, B * 8 + 5
            self.table = torch.randperm(blocks, generator=g)[:B * 8].view(B, 8).int().cuda()
            self.entry = self.table.cpu().long()[rows, self.at // page] * page + self.at % page
            total = blocks * page
        elif layout == "contiguous":
            blocks, total = 0, B * room
            self.entry = rows * room + self.at
        else:
            blocks = total = B * room + 3
            self.entry = rows = torch.randperm(blocks, generator=g)[:n]
        self.total, self.rows = total, rows.int().cuda()
        self.entries = self.at.int().cuda() if entries and layout != "indexed" else None
        self.prob = api.problem(batch=B, num_q_heads=H_q, num_kv_heads=H, head_dim_qk=D, layout=layout, scale=0.1,
                                page_size=page if layout == "paged" else 0, width=width, num_blocks=blocks,
                                kv_dtype=KV.index(kv), k_scale=K_SCALE, v_scale=V_SCALE)
        m = total * H * D
        size = {"bf16": 2 * m, "e4m3": m, "nvfp4": m // 2 + m // 16}[kv]
        self.before = [torch.randint(0, 256, (size,), generator=g, dtype=torch.int32).to(torch.uint8).cuda()
                       for _ in range(2)]
        self.caches = [t.clone() for t in self.before]
        wt = torch.bfloat16 if w == "bf16" else torch.float32
        self.qw, self.kw = ((torch.randn(D, generator=g) * 0.3 + 1 - w_add).to(wt).cuda() if c in which else None
                            for c in "qk")
        self.norm = api.head_norm(self.qw, self.kw, eps=eps, w_add=w_add)
        self.spec, self.inv, self.rope = rope, None, None
        if rope:
            self.inv = (10000.0 ** (-torch.arange(rope[0] // 2, dtype=torch.float64) * 2 / rope[0])).float()
            self.rope = api.rope(self.inv.cuda(), offset=rope[1], interleaved=rope[2])

    def run(self, api, **kw):
        k, v = ((t.view(torch.bfloat16) if self.kv == "bf16" else t) for t in self.caches)
        kw.setdefault("rows", self.rows)
        kw.setdefault("entries", self.entries)
        kw.setdefault("q_new", self.q)
        pos = kw.pop("positions") if "positions" in kw else self.pos.int().cuda()
        return api.append(self.prob, self.rope, self.k_new, self.v_new, k, v, pos, table=self.table, norm=self.norm, **kw)

    def want(self, x, w):
        """(values, error bound) of normed and rotated heads, fp64."""
        x = x.double().cpu().numpy()
        fuzz = np.zeros_like(x)
        if w is not None:
            x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + self.eps) * (w.double().cpu().numpy() + self.w_add)
            fuzz = 2.0 ** -19 * np.abs(x)
        if not self.spec:
            return x, fuzz
        dim, off, inter = self.spec
        mag = np.abs(x)
        part = mag[..., off:off + dim]
        other = (part.reshape(*part.shape[:-1], dim // 2, 2)[..., ::-1].reshape(part.shape) if inter else
                 np.concatenate([part[..., dim // 2:], part[..., :dim // 2]], -1))
        fuzz[..., off:off + dim] = 2.0 ** -18 * (part + other)
        return OS.rotate(x, self.pos.numpy(), self.inv.numpy(), off, inter), fuzz

    def check(self, q, live=None):
        live = np.arange(self.n) if live is None else live
        if q is not None:
            ref, fuzz = self.want(self.q, self.qw)
            err = np.abs(q.double().cpu().numpy() - ref)[live]
            assert np.all(err <= (2.0 ** -8 * np.abs(ref) + fuzz)[live])
        H, D = self.heads[1:]
        entry = self.entry.numpy()[live]
        for i, (new, w, scale) in enumerate(((self.k_new, self.kw, K_SCALE), (self.v_new, None, V_SCALE))):
            ref, fuzz = self.want(new, w) if i == 0 else (new.double().cpu().numpy(), np.zeros(new.shape))
            ref, fuzz = ref[live], fuzz[live]
            after, before = self.caches[i].cpu().numpy(), self.before[i].cpu().numpy()
            m = self.total * H * D
            if self.kv == "bf16":
                parts = [(after, before, 2 * H * D)]
                got = torch.from_numpy(after).view(torch.bfloat16).double().numpy().reshape(-1, H, D)[entry]
                tol = 2.0 ** -8 * np.abs(ref) + fuzz
            elif self.kv == "e4m3":
                parts = [(after, before, H * D)]
                got = OF.decode_e4m3(after).reshape(-1, H, D)[entry] * scale
                ref = np.clip(ref, -448 * scale, 448 * scale)
                tol = 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * scale + fuzz
            else:
                parts = [(after[:m // 2], before[:m // 2], H * D // 2), (after[m // 2:], before[m // 2:], H * D // 16)]
                s = OF.decode_e4m3(after[m // 2:]).reshape(-1, H, D // 16)[entry]
                blocks = ref.reshape(*ref.shape[:-1], D // 16, 16)
                f16 = fuzz.reshape(blocks.shape).max(-1)
                want = np.minimum(np.abs(blocks).max(-1) / (6 * scale), 448)
                assert np.all(np.abs(s - want) <= 2.0 ** -4 * want + 2.0 ** -10 + f16 / (6 * scale))
                step = np.repeat(s, 16, -1) * scale
                got = ON.decode_e2m1(ON.unpack(after[:m // 2].reshape(-1, H, D // 2)[entry])) * step
                a = np.minimum(np.abs(ref), 6 * step)
                half = np.where(a > 4 * step, 1.0, np.where(a > 2 * step, 0.5, 0.25)) * step
                ref = np.clip(ref, -6 * step, 6 * step)
                tol = half * (1 + 2.0 ** -20) + fuzz + 2.0 ** -20 * np.abs(ref)
            assert np.all(np.abs(got - ref) <= tol), i
            for a, b, size in parts:  # nothing else has changed
                a, b = a.reshape(-1, size).copy(), b.reshape(-1, size)
                a[entry] = b[entry]
                assert np.array_equal(a, b)


# (layout, kv, heads, rope (dim, offset, interleaved), x, w, w_add, which, n)
GRID = [
    ("paged", "bf16", (8, 2, 128), (128, 0, False), "bf16", "bf16", 0.0, "qk", 1),
    ("paged", "bf16", (8, 2, 128), (128, 0, True), "fp32", "fp32", 1.0, "qk", 37),
    ("contiguous", "bf16", (3, 3, 64), (64, 0, False), "fp32", "bf16", 0.0, "k", 5),
    ("indexed", "bf16", (32, 8, 128), (32, 96, False), "bf16", "fp32", 0.0, "q", 130),
    ("paged", "e4m3", (8, 2, 128), (64, 64, True), "bf16", "bf16", 0.0, "qk", 64),
    ("contiguous", "e4m3", (12, 4, 64), None, "fp32", "fp32", 0.0, "qk", 33),
    ("paged", "nvfp4", (8, 2, 128), (128, 0, False), "bf16", "bf16", 0.0, "qk", 51),
    ("contiguous", "nvfp4", (7, 1, 64), (16, 8, True), "fp32", "bf16", 1.0, "qk", 2),
    ("indexed", "nvfp4", (16, 4, 64), (48, 16, False), "bf16", "fp32", 0.0, "k", 400),
    ("paged", "nvfp4", (20, 4, 64), (32, 32, False), "fp32", "fp32", 0.0, "qk", 300),
]


@gpu
@pytest.mark.parametrize("layout,kv,heads,rope,x,w,w_add,which,n", GRID)
def test_against_fp64(api, layout, kv, heads, rope, x, w, w_add, which, n):
    c = Case(api, layout=layout, kv=kv, heads=heads, rope=rope, x=x, w=w, w_add=w_add, which=which, n=n, seed=n)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = c.run(api, err=err)
    assert int(err) == 0
    c.check(q)


@gpu
@pytest.mark.parametrize("kv", KV)
def test_many_tokens(api, kv):
    c = Case(api, n=1500, kv=kv, heads=(32, 8, 128), page=64, seed=1)
    c.check(c.run(api))


@gpu
def test_entries_without_norms_store_what_a_plain_append_does(api):
    """A token rotated by one position and stored at another entry has the bytes that
    an append of that position leaves."""
    c = Case(api, entries=False, seed=2)
    plain = [t.clone() for t in c.before]
    views = [t.view(torch.bfloat16) for t in plain]
    q1 = api.append(c.prob, c.rope, c.k_new, c.v_new, *views, c.pos.int().cuda(), rows=c.rows, table=c.table, q_new=c.q)
    flip = (128 - 1 - c.at).int()  # the same positions, entries in reverse
    moved = [t.clone() for t in c.before]
    views = [t.view(torch.bfloat16) for t in moved]
    q2 = api.append(c.prob, c.rope, c.k_new, c.v_new, *views, c.pos.int().cuda(), rows=c.rows, table=c.table, q_new=c.q,
                    entries=flip.cuda())
    assert torch.equal(q1, q2)
    rows, table = c.rows.cpu().long(), c.table.cpu().long()
    to = table[rows, flip.long() // 16] * 16 + flip.long() % 16
    for a, b in zip(plain, moved):
        a, b = a.view(-1, 512), b.view(-1, 512)
        assert torch.equal(a[c.entry.cuda()], b[to.cuda()])


@gpu
def test_a_token_depends_on_itself_alone(api):
    big = Case(api, n=300, kv="nvfp4", page=16, seed=3)
    q = big.run(api)
    for i in (0, 7, 299):
        k, v = (t.clone() for t in big.before)
        one = api.append(big.prob, big.rope, big.k_new[i:i + 1], big.v_new[i:i + 1], k, v, big.pos[i:i + 1].int().cuda(),
                         rows=big.rows[i:i + 1], table=big.table, q_new=big.q[i:i + 1], norm=big.norm,
                         entries=big.entries[i:i + 1])
        assert torch.equal(one[0], q[i])
        m = big.total * 2 * 128
        at = int(big.entry[i])
        for a, b in ((k, big.caches[0]), (v, big.caches[1])):
            assert torch.equal(a[:m // 2].view(-1, 128)[at], b[:m // 2].view(-1, 128)[at])
            assert torch.equal(a[m // 2:].view(-1, 16)[at], b[m // 2:].view(-1, 16)[at])


@gpu
def test_special_rows(api):
    c = Case(api, n=6, x="fp32", heads=(2, 1, 64), rope=None, seed=4)
    c.q[0] = 0                     # a zero head stays zero
    c.q[1, 0, 3] = float("nan")    # spoils its head alone
    c.q[2, 1, 5] = float("inf")
    c.q[3] = 1e-20                 # below eps: nearly zero
    c.q[4] = 1e15                  # far above it
    q = c.run(api).float().cpu()
    ref = c.want(c.q, c.qw)[0]
    assert (q[0] == 0).all()
    assert q[1, 0].isnan().all() and torch.isfinite(q[1, 1]).all()
    assert q[2, 1, 5].isnan() and (q[2, 1, [0, 1, 2, 3, 4, 6]] == 0).all() and torch.isfinite(q[2, 0]).all()
    for i in (3, 4, 5):
        assert np.all(np.abs(q[i].numpy() - ref[i]) <= 2.0 ** -8 * np.abs(ref[i]) + 2.0 ** -18 * np.abs(ref[i]))


@gpu
def test_padded_and_bad_tokens(api):
    c = Case(api, n=12, seed=5)
    rows, entries = c.rows.clone(), c.entries.clone()
    rows[1] = -1
    entries[3], entries[5] = -1, 128  # beyond the capacity
    pos = c.pos.int().cuda()
    pos[8] = -4
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.full((12, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    c.run(api, rows=rows, entries=entries, positions=pos, err=err, q_out=q)
    assert int(err) == api.DEVERR_LENGTH
    left = [1, 3, 5, 8]
    assert (q[left] == 3.0).all()
    c.check(q, live=np.array([i for i in range(12) if i not in left]))


@gpu
def test_streams_and_graphs(api):
    c = Case(api, n=40, kv="e4m3", seed=6)
    want, q_want = c.run(api).clone(), [t.clone() for t in c.caches]
    s = torch.cuda.Stream()
    for t, b in zip(c.caches, c.before):
        t.copy_(b)
    torch.cuda.synchronize()
    q = c.run(api, stream=s)
    s.synchronize()
    assert torch.equal(q, want) and all(torch.equal(a, b) for a, b in zip(c.caches, q_want))
    graph, out, pos = torch.cuda.CUDAGraph(), torch.zeros_like(want), c.pos.int().cuda()
    with torch.cuda.graph(graph):
        c.run(api, q_out=out, positions=pos)
    for t, b in zip(c.caches, c.before):
        t.copy_(b)
    c.pos = (c.pos * 7 + 1) % 4999
    pos.copy_(c.pos.int())
    graph.replay()
    c.check(out)


def packed(api, **kw):
    a = dict(n=2, x=api.X_BF16, k_new=1 << 20, v_new=1 << 21, q_new=1 << 22, ks=256, vs=256, qs=1024, pos=1 << 23,
             rows=1 << 24, table=1 << 25, k=1 << 26, v=1 << 27, q_out=1 << 28, err=0)
    a.update(kw)
    return api._APPEND.pack(*a.values())


def test_argument_rules(api):
    L = api.lib()
    prob = api.problem(batch=2, num_q_heads=8, num_kv_heads=2, head_dim_qk=128, layout="paged", scale=0.1, page_size=16,
                       width=8, num_blocks=20)
    base = dict(q_weight=1 << 12, k_weight=1 << 13, w_dtype=api.X_BF16, w_add=0.0, eps=1e-6)

    def call(p=prob, args=None, entries=None, **kw):
        n = api.DaHeadNorm(*{**base, **kw}.values())
        return L.decode_attn_append_norm(ctypes.addressof(p), None, ctypes.addressof(n), args or packed(api), entries, None)

    inv, uns = api.ERR_INVALID_ARG, api.ERR_UNSUPPORTED
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(w_add=float("inf")), dict(w_dtype=7),
               dict(q_weight=(1 << 12) + 8), dict(k_weight=(1 << 13) + 2), dict(entries=(1 << 14) + 2),
               dict(args=packed(api, q_new=0, q_out=0)), dict(args=packed(api, n=-1)), dict(args=packed(api, pos=0))):
        assert call(**kw) == inv, kw
    assert L.decode_attn_append_norm(None, None, None, packed(api), None, None) == inv
    assert L.decode_attn_append_norm(ctypes.addressof(prob), None, None, None, None, None) == inv
    slots = api.problem(batch=2, num_q_heads=8, num_kv_heads=2, head_dim_qk=128, layout="indexed", scale=0.1, width=8,
                        num_blocks=20)
    assert call(p=slots, entries=1 << 14) == inv  # slots are in rows already
    latent = api.problem(batch=2, num_q_heads=16, num_kv_heads=1, head_dim_qk=576, head_dim_v=512, layout="paged",
                         scale=0.1, page_size=16, width=8, num_blocks=20, shared_latent=True)
    assert call(p=latent, args=packed(api, v_new=0, v=0, ks=576, qs=16 * 576)) == uns
    assert call(args=packed(api, n=0)) == api.OK


def test_queries_over_weights_or_entries(api):
    """What the threads of every token read is not to be written by any of them."""
    prob = api.problem(batch=2, num_q_heads=8, num_kv_heads=2, head_dim_qk=128, layout="paged", scale=0.1, page_size=16,
                       width=8, num_blocks=20)
    q_out, end = 1 << 28, (1 << 28) + 2 * 8 * 128 * 2

    def call(dtype=api.X_BF16, entries=0, q_weight=1 << 12, k_weight=1 << 13):
        n = api.DaHeadNorm(q_weight, k_weight, dtype, 0.0, 1e-6)
        return api.lib().decode_attn_append_norm(ctypes.addressof(prob), None, ctypes.addressof(n), packed(api),
                                                 entries or None, None)

    over = [dict(q_weight=q_out), dict(k_weight=end - 16), dict(q_weight=q_out - 256 + 16),
            dict(dtype=api.X_F32, k_weight=q_out - 512 + 16), dict(entries=end - 4), dict(entries=q_out - 4),
            dict(entries=q_out + 64)]
    for kw in over:
        assert call(**kw) == api.ERR_INVALID_ARG, kw
    if not torch.cuda.is_available():  # (the addresses are no one's)
        for kw in (dict(), dict(q_weight=end), dict(k_weight=q_out - 256), dict(entries=q_out - 8), dict(entries=end)):
            assert call(**kw) == api.ERR_CUDA, kw


def test_python_checks(api):
    w = torch.ones(128)
    with pytest.raises(ValueError, match="needs"):
        api.head_norm(eps=1e-6)
    with pytest.raises(ValueError, match="vectors"):
        api.head_norm(torch.ones(128, dtype=torch.float64), eps=1e-6)
    with pytest.raises(ValueError, match="k_weight"):
        api.head_norm(w, w.bfloat16(), eps=1e-6)
    with pytest.raises(ValueError, match="k_weight"):
        api.head_norm(w, w[:64].clone(), eps=1e-6)
    prob = api.problem(batch=2, num_q_heads=2, num_kv_heads=1, head_dim_qk=64, layout="contiguous", scale=0.1, width=8)
    k_new, cache = torch.zeros((2, 1, 64)), torch.zeros((2, 8, 1, 64), dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="128 elements"):
        api.append(prob, None, k_new, k_new.clone(), cache, cache.clone(), pos, norm=api.head_norm(None, w, eps=1e-6))
    with pytest.raises(ValueError, match="entries"):
        api.append(prob, None, k_new, k_new.clone(), cache, cache.clone(), pos, entries=pos.long())
    with pytest.raises(ValueError, match="no CPU path"):
        api.append(prob, None, k_new, k_new.clone(), cache, cache.clone(), pos, entries=pos)
