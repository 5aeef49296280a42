"""decode_attn_append: new keys and values into the caches that attention
reads, keys and queries rotated, against the fp64 oracle.

Tolerance.  The rotated value is v = a cos +- b sin in fp32: the angle's own
rounding (2^-23), sin and cos (2^-23), two products and a sum (2^-24 each) leave
an error below 2^-20 (|a| + |b|).  Storing rounds once, by at most half a step:
2^-8 of the value for bf16, 2^-4 for E4M3 (and 2^-10 of the scale where E4M3 has
no smaller step), half the spacing of the eight E2M1 magnitudes for NVFP4.
What is copied and not rotated has no fp32 error: its bytes are compared with
the same operations of torch, bit for bit."""

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
    """Random projections, a cache with contents, and where each token goes."""

    def __init__(self, api, *, n, layout="paged", kv="bf16", heads=(8, 2, 128), rope=None, x="bf16",
                 page=16, B=4, fused=True, latent=False, seed=0, gain=1.0, positions=None):
        g = torch.Generator().manual_seed(seed)
        H_q, H_kv, D = heads
        self.kv, self.heads, self.n, self.latent, self.layout = kv, heads, n, latent, layout
        dt = torch.bfloat16 if x == "bf16" else torch.float32
        if latent or not fused:
            q = torch.randn((n, H_q, D), generator=g).to(dt)
            k = torch.randn((n, H_kv, D), generator=g).to(dt)
            v = None if latent else torch.randn((n, H_kv, D), generator=g).to(dt)
            self.q, self.k_new, self.v_new = (None if t is None else t.cuda() for t in (q, k, v))
        else:  # parts of one projection's rows
            row = torch.randn((n, (H_q + 2 * H_kv) * D), generator=g).to(dt).cuda()
            self.q = row[:, :H_q * D].view(n, H_q, D)
            self.k_new = row[:, H_q * D:(H_q + H_kv) * D].view(n, H_kv, D)
            self.v_new = row[:, (H_q + H_kv) * D:].view(n, H_kv, D)
        width = 8 if layout == "paged" else 8 * page
        room = 8 * page
        pick = torch.randperm(B * room, generator=g)[:n]
        self.rows, self.pos = pick // room, pick % room
        self.table = None
        if layout == "paged":
            blocks = B * 8 + 5
            self.table = torch.randperm(blocks, generator=g)[:B * 8].view(B, 8).int()
            self.entry = (self.table.long()[self.rows, self.pos // page] * page + self.pos % page)
            self.total = blocks * page
        elif layout == "contiguous":
            blocks, self.total = 0, B * room
            self.entry = self.rows * room + self.pos
        else:
            blocks = self.total = B * room + 3
            self.entry = torch.randperm(blocks, generator=g)[:n]
            self.rows = self.entry
        if positions is not None:
            self.pos = torch.as_tensor(positions)
        self.prob = api.problem(batch=B, num_q_heads=H_q, num_kv_heads=H_kv, head_dim_qk=D,
                                head_dim_v=512 if latent else D, layout=layout, scale=0.1,
                                page_size=page if layout == "paged" else 0, width=width,
                                num_blocks=blocks, shared_latent=latent,
                                kv_dtype=KV.index(kv), k_scale=K_SCALE, v_scale=V_SCALE)
        m = self.total * H_kv * D
        size = {"bf16": 2 * m, "e4m3": m, "nvfp4": m // 2 + m // 16}[kv]
        self.before = [torch.randint(0, 256, (size,), generator=g, dtype=torch.int32)
                       .to(torch.uint8).cuda() for _ in range(1 if latent else 2)]
        self.caches = [t.clone() for t in self.before]
        view = (lambda t: t.view(torch.bfloat16)) if kv == "bf16" else (lambda t: t)
        self.k = view(self.caches[0])
        self.v = None if latent else view(self.caches[1])
        self.spec, self.gain, self.rope, self.inv = rope, gain, None, None
        if rope is not None:
            dim, off, inter = rope
            self.inv = (10000.0 ** (-torch.arange(dim // 2, dtype=torch.float64) * 2 / dim)).float()
            self.rope = api.rope(self.inv.cuda(), offset=off, interleaved=inter, gain=gain)

    def i32(self, t):
        return None if t is None else t.to(torch.int32).cuda()

    def run(self, api, **kw):
        kw.setdefault("rows", self.i32(self.rows))
        kw.setdefault("positions", self.i32(self.pos))
        if "q_new" not in kw:
            kw["q_new"] = self.q
        pos = kw.pop("positions")
        return api.append(self.prob, self.rope, self.k_new, self.v_new, self.k, self.v, pos,
                          table=self.i32(self.table), **kw)

    def turned(self, x):
        """(exact rotated values, magnitudes |a| + |b|) as fp64."""
        x = x.double().cpu().numpy()
        if self.spec is None:
            return x, np.zeros_like(x)
        dim, off, inter = self.spec
        mag = np.abs(x)
        part = mag[..., off:off + dim]
        other = (part.reshape(*part.shape[:-1], dim // 2, 2)[..., ::-1].reshape(part.shape) if inter
                 else np.concatenate([part[..., dim // 2:], part[..., :dim // 2]], -1))
        fuzz = np.zeros_like(x)
        fuzz[..., off:off + dim] = (part + other) * abs(self.gain)
        return OS.rotate(x, self.pos.numpy(), self.inv.numpy(), off, inter, self.gain), fuzz

    def check_q(self, q, live=None):
        live = np.arange(self.n) if live is None else live
        ref, fuzz = self.turned(self.q)
        err = np.abs(q.double().cpu().numpy() - ref)[live]
        assert np.all(err <= (2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * fuzz)[live]), err.max()

    def check_caches(self, live=None):
        live = np.arange(self.n) if live is None else live
        H, D = self.heads[1:]
        entry = self.entry.numpy()[live]
        for i, (new, scale) in enumerate([(self.k_new, K_SCALE), (self.v_new, V_SCALE)][
                :len(self.caches)]):
            after, before = self.caches[i].cpu().numpy(), self.before[i].cpu().numpy()
            ref, fuzz = (self.turned(new) if i == 0 else
                         (new.double().cpu().numpy(), np.zeros(new.shape)))
            ref, fuzz = ref[live], 2.0 ** -20 * fuzz[live]
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
                m = self.total * H * D
                parts = [(after[:m // 2], before[:m // 2], H * D // 2),
                         (after[m // 2:], before[m // 2:], H * D // 16)]
                codes = after[:m // 2].reshape(-1, H, D // 2)[entry]
                s = OF.decode_e4m3(after[m // 2:]).reshape(-1, H, D // 16)[entry]
                blocks = ref.reshape(*ref.shape[:-1], D // 16, 16)
                f16 = fuzz.reshape(blocks.shape).max(-1)
                want = np.minimum(np.abs(blocks).max(-1) / (6 * scale), 448)
                assert np.all(np.abs(s - want) <= 2.0 ** -4 * want + 2.0 ** -10 + f16 / (6 * scale))
                step = np.repeat(s, 16, -1) * scale
                got = ON.decode_e2m1(ON.unpack(codes)) * step
                a = np.minimum(np.abs(ref), 6 * step)
                half = np.where(a > 4 * step, 1.0, np.where(a > 2 * step, 0.5, 0.25)) * step
                ref = np.clip(ref, -6 * step, 6 * step)
                # (1 + 2^-20): the fp32 division by the step
                tol = half * (1 + 2.0 ** -20) + fuzz + 2.0 ** -20 * np.abs(ref)
            err = np.abs(got - ref)
            assert np.all(err <= tol), (i, float((err - tol).max()))
            for a, b, size in parts:  # nothing else has changed
                a, b = a.reshape(-1, size).copy(), b.reshape(-1, size)
                a[entry] = b[entry]
                assert np.array_equal(a, b)


# (layout, kv, heads, rope (dim, offset, interleaved), x, n, fused)
GRID = [
    ("paged", "bf16", (8, 2, 128), (128, 0, False), "bf16", 1, True),
    ("paged", "bf16", (8, 2, 128), (128, 0, True), "fp32", 37, True),
    ("contiguous", "bf16", (3, 3, 64), (64, 0, False), "fp32", 5, False),
    ("indexed", "bf16", (32, 8, 128), (32, 96, False), "bf16", 130, True),
    ("paged", "e4m3", (8, 2, 128), (64, 64, True), "bf16", 64, True),
    ("contiguous", "e4m3", (12, 4, 64), (64, 0, False), "fp32", 33, True),
    ("indexed", "e4m3", (128, 8, 128), (128, 0, False), "fp32", 3, True),
    ("paged", "nvfp4", (8, 2, 128), (128, 0, False), "bf16", 51, True),
    ("contiguous", "nvfp4", (7, 1, 64), (16, 8, True), "fp32", 2, False),
    ("indexed", "nvfp4", (16, 4, 64), (48, 16, False), "bf16", 400, True),
    ("paged", "bf16", (5, 5, 64), None, "fp32", 400, True),
    ("paged", "nvfp4", (20, 4, 64), None, "fp32", 9, True),
]


@gpu
@pytest.mark.parametrize("layout,kv,heads,rope,x,n,fused", GRID)
def test_against_oracle(api, layout, kv, heads, rope, x, n, fused):
    c = Case(api, n=n, layout=layout, kv=kv, heads=heads, rope=rope, x=x, fused=fused, seed=n,
             gain=1.25 if rope and rope[2] else 1.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = c.run(api, err=err)
    assert int(err) == 0
    c.check_q(q)
    c.check_caches()


@gpu
@pytest.mark.parametrize("page", [1, 3, 64])
def test_page_sizes(api, page):
    c = Case(api, n=20, kv="e4m3", rope=(128, 0, False), page=page, seed=page)
    c.check_q(c.run(api))
    c.check_caches()


@gpu
@pytest.mark.parametrize("kv,n,inter", [("bf16", 1, True), ("e4m3", 5, False), ("bf16", 330, True)])
def test_shared_latent(api, kv, n, inter):
    c = Case(api, n=n, layout="indexed", kv=kv, heads=(16, 1, 576), rope=(64, 512, inter),
             latent=True, seed=n)
    c.check_q(c.run(api))
    c.check_caches()


@gpu
@pytest.mark.parametrize("x", ["bf16", "fp32"])
def test_many_tokens_use_wide_parts(api, x):
    c = Case(api, n=900, kv="nvfp4", heads=(32, 8, 128), rope=(128, 0, False), x=x, B=9, page=16)
    c.check_q(c.run(api))
    c.check_caches()


@gpu
def test_far_positions(api):
    # any position may rotate an indexed cache's keys; angles up to 2^31 radians
    pos = [0, 1, 4095, 131071, 1 << 20, (1 << 24) + 1, (1 << 30) + 12345, (1 << 31) - 1]
    c = Case(api, n=8, layout="indexed", rope=(128, 0, False), x="fp32", positions=pos)
    c.check_q(c.run(api))
    c.check_caches()


@gpu
@pytest.mark.parametrize("inter", [False, True])
def test_sine_and_cosine_have_fp32_accuracy(api, inter):
    """A vector (sin t, cos t) turned by t has a first component near zero, whose bf16
    bits show the absolute error of the rotation that a result of ordinary size hides.

    With |a|, |b| <= 1 and a sin t + b cos t = 1: the angle is rounded once to fp32, in
    half turns of at most 1 (2^-25 of them: 0.80 * 2^-23 in radians); sine and
    cosine are off by two units of 2^-24 at most, together sqrt(2) * 2^-23; the two products
    of magnitude at most 1/2 by 2^-26 each.  Sum: 2.47 * 2^-23 < 1.25 * 2^-22."""
    g = torch.Generator().manual_seed(5)
    n, half = 64, 64
    pos = torch.randint(0, 1 << 17, (n,), generator=g)
    inv = torch.exp2(-13 * torch.rand(half, generator=g, dtype=torch.float64)).float()
    t = pos.double().numpy().astype(np.longdouble)[:, None] * inv.numpy().astype(np.longdouble)
    x = np.zeros((n, 1, 2 * half))
    ia = 2 * np.arange(half) if inter else np.arange(half)
    ib = ia + (1 if inter else half)
    x[:, 0, ia], x[:, 0, ib] = np.sin(t), np.cos(t)
    q = torch.from_numpy(x).float()
    prob = api.problem(batch=1, num_q_heads=1, num_kv_heads=1, head_dim_qk=128, layout="indexed",
                       scale=0.1, width=1, num_blocks=n)
    k, v = (torch.zeros((n, 1, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    out = api.append(prob, api.rope(inv.cuda(), interleaved=inter), q.cuda(), q.cuda(), k, v,
                     pos.to(**i32), rows=torch.arange(n, **i32), q_new=q.cuda())
    ref = OS.rotate(q.double().numpy(), pos.numpy(), inv.numpy(), interleaved=inter)
    tol = 2.0 ** -8 * np.abs(ref) + 1.25 * 2.0 ** -22
    for got in (out, k):
        err = np.abs(got.double().cpu().numpy() - ref)[:, 0, ia]
        assert np.all(err <= tol[:, 0, ia]), float(err.max() * 2 ** 22)


@gpu
def test_angles_far_beyond_32_bits(api):
    # the product of a position and a frequency is exact, whatever the frequency
    pos = [1, 4095, (1 << 24) + 1, (1 << 30) + 12345, (1 << 31) - 1, (1 << 31) - 77]
    c = Case(api, n=6, layout="indexed", rope=(128, 0, False), x="fp32", positions=pos)
    c.inv = torch.exp2(torch.linspace(-4, 18, 64, dtype=torch.float64)).float()
    c.inv[1::3] *= -1
    c.rope = api.rope(c.inv.cuda())
    c.check_q(c.run(api))
    c.check_caches()


@gpu
@pytest.mark.parametrize("kv", KV)
def test_prompts_of_many_tokens(api, kv):
    c = Case(api, n=1500, kv=kv, heads=(20, 4, 128), rope=(96, 16, False), x="bf16", B=12, page=16,
             seed=15)
    c.check_q(c.run(api))
    c.check_caches()


@gpu
def test_frequencies_at_the_ends_of_their_range(api):
    # denormal and tiny ones turn by nothing, zero by nothing at all, in both directions
    c = Case(api, n=5, layout="indexed", rope=(128, 0, True), x="fp32",
             positions=[0, 1, 7, 1 << 20, (1 << 31) - 1])
    c.inv = torch.cat([torch.tensor([0.0, -0.0, 1e-45, -1e-40, 2.0 ** -126, 2.0 ** -100, -(2.0 ** -64)]),
                       torch.exp2(torch.linspace(-60, 17, 57, dtype=torch.float64)).float()])
    c.rope = api.rope(c.inv.cuda(), interleaved=True)
    c.check_q(c.run(api))
    c.check_caches()


@gpu
@pytest.mark.parametrize("kv", KV)
def test_entries_beyond_32_bits(api, kv):
    """A cache of more than 2^32 elements: entries at both ends and around 2^31 and 2^32
    elements get what the same tokens get in a small cache."""
    n, H_kv, D = 7, 8, 128
    slots = (1 << 22) + 5  # 1024 elements each
    at = torch.tensor([0, (1 << 21) - 1, 1 << 21, (1 << 22) - 1, 1 << 22, slots - 2, slots - 1])
    g = torch.Generator().manual_seed(7)
    k_new, v_new = (torch.randn((n, H_kv, D), generator=g).cuda() for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    rope = api.rope(torch.rand(64, generator=g).cuda())
    got = []
    for count, rows in ((n, torch.arange(n)), (slots, at)):
        prob = api.problem(batch=1, num_q_heads=H_kv, num_kv_heads=H_kv, head_dim_qk=D, layout="indexed",
                           scale=0.1, width=1, num_blocks=count, kv_dtype=KV.index(kv), k_scale=K_SCALE,
                           v_scale=V_SCALE)
        m = count * H_kv * D
        size = {"bf16": 2 * m, "e4m3": m, "nvfp4": m // 2 + m // 16}[kv]
        pair = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
        k, v = (t.view(torch.bfloat16) if kv == "bf16" else t for t in pair)
        api.append(prob, rope, k_new, v_new, k, v, torch.arange(n, **i32), rows=rows.to(**i32))
        for t in pair:
            parts = [t[:m // 2], t[m // 2:]] if kv == "nvfp4" else [t]
            got.append([p.view(count, -1)[rows.cuda()] for p in parts])
            written = sum(int(torch.count_nonzero(p.view(count, -1).view(torch.int32).any(1)))
                          for p in parts)
            assert written == n * len(parts)
        del pair, k, v, t, parts
    torch.cuda.empty_cache()
    for small, large in ((got[0], got[2]), (got[1], got[3])):
        assert all(torch.equal(a, b) for a, b in zip(small, large))


@gpu
@pytest.mark.parametrize("x", ["bf16", "fp32"])
def test_copied_values_are_stored_like_torch_stores_them(api, x):
    """Without a rotation the stored bytes are those of torch's conversions."""
    for kv in KV:
        c = Case(api, n=30, kv=kv, x=x, seed=5)
        for t in (c.k_new, c.v_new):  # spread the magnitudes, cross saturation
            t.mul_(torch.exp2(torch.randint(-12, 5, t.shape, device="cuda").float()).to(t.dtype))
        q = c.run(api)
        assert torch.equal(q, c.q.to(torch.bfloat16))
        H, D = c.heads[1:]
        e = c.entry.cuda()
        for new, cache, scale in ((c.k_new, c.caches[0], K_SCALE), (c.v_new, c.caches[1], V_SCALE)):
            f, scale = new.float(), torch.tensor(scale, device="cuda")
            if kv == "bf16":
                got = cache.view(torch.bfloat16).view(-1, H, D)[e]
                assert torch.equal(got, f.to(torch.bfloat16))
            elif kv == "e4m3":
                want = (f / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                assert torch.equal(cache.view(-1, H, D)[e], want)
            else:
                m = c.total * H * D
                b = f.view(c.n, H, D // 16, 16)
                want = (b.abs().amax(-1) / (scale * 6)).clamp(max=448).to(torch.float8_e4m3fn)
                s = cache[m // 2:].view(-1, H, D // 16)[e]
                assert torch.equal(s, want.view(torch.uint8))
                step = (want.float() * scale)[..., None]
                u = torch.where(step > 0, b / step, torch.zeros_like(b)).double().cpu().numpy()
                mag = OS._nearest(np.abs(u), OS._E2M1) | np.where(np.signbit(u), 8, 0)
                mag = mag.reshape(c.n, H, D)
                packed = (mag[..., 0::2] | mag[..., 1::2] << 4).astype(np.uint8)
                got = cache[:m // 2].view(-1, H, D // 2)[e].cpu().numpy()
                assert np.array_equal(got, packed)


@gpu
def test_special_values(api):
    """NaN, infinities and zeros end up where they belong and nowhere else."""
    nan, inf = float("nan"), float("inf")
    for kv in KV:
        c = Case(api, n=4, kv=kv, x="fp32", fused=False, seed=9)
        c.v_new[0, 0, 3] = nan
        c.v_new[1, 0, 20] = inf
        c.v_new[2, 1, :] = 0
        c.v_new[3, 0, 16:32] = 1e-30  # below every block scale
        c.run(api)
        H, D = c.heads[1:]
        e = c.entry.cuda()
        if kv == "bf16":
            got = c.v.view(-1, H, D)[e].float()
            assert torch.isnan(got).sum() == 1 and torch.isnan(got[0, 0, 3])
            assert got[1, 0, 20] == inf
        elif kv == "e4m3":
            got = OF.decode_e4m3(c.v.view(-1, H, D)[e].cpu().numpy())
            assert np.isnan(got).sum() == 1 and np.isnan(got[0, 0, 3])
            assert got[1, 0, 20] == 448 and np.all(got[2, 1] == 0) and np.all(got[3, 0, 16:32] == 0)
        else:
            m = c.total * H * D
            codes = c.v[:m // 2].view(-1, H, D // 2)[e].cpu().numpy()
            s = OF.decode_e4m3(c.v[m // 2:].view(-1, H, D // 16)[e].cpu().numpy())
            assert np.isnan(s).sum() == 1 and np.isnan(s[0, 0, 0])  # the NaN's block
            val = ON.decode_e2m1(ON.unpack(codes))
            assert s[1, 0, 1] == 448 and val[1, 0, 20] == 6
            assert np.all(s[2, 1] == 0) and np.all(val[2, 1] == 0)
            assert s[3, 0, 1] == 0 and np.all(val[3, 0, 16:32] == 0)


@gpu
def test_padding_and_out_of_range_tokens_write_nothing(api):
    for layout in ("paged", "contiguous", "indexed"):
        c = Case(api, n=12, layout=layout, rope=(128, 0, False), seed=3)
        rows, pos = c.rows.clone(), c.pos.clone()
        rows[1] = -1
        rows[2] = -(1 << 31)
        rows[4] = c.total if layout == "indexed" else c.prob.batch
        pos[6] = -1
        bad = [1, 2, 4, 6]
        if layout != "indexed":
            pos[7] = 8 * 16
            bad.append(7)
        if layout == "paged":
            c.table[rows[9], pos[9] // 16] = -1
            hit = [i for i in range(12) if i not in bad and rows[i] == rows[9]
                   and pos[i] // 16 == pos[9] // 16]
            bad += hit
        live = np.array([i for i in range(12) if i not in bad])
        q = torch.full((12, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.run(api, rows=c.i32(rows), positions=c.i32(pos), q_out=q, err=err)
        assert int(err) == api.DEVERR_LENGTH | api.DEVERR_INDEX
        assert torch.all(q[bad] == 7)
        c.check_q(q, live)
        c.check_caches(live)
        # bits are OR-ed in and padding alone sets none
        err.fill_(api.DEVERR_TIMEOUT)
        c.run(api, rows=torch.full((12,), -1, dtype=torch.int32, device="cuda"), err=err)
        assert int(err) == api.DEVERR_TIMEOUT


@gpu
def test_rows_default_no_queries_and_no_error_word(api):
    c = Case(api, n=4, rope=(128, 0, False), seed=11)
    c.rows = torch.arange(4)
    c.entry = c.table.long()[c.rows, c.pos // 16] * 16 + c.pos % 16
    assert c.run(api, rows=None, q_new=None) is None
    c.check_caches()


@gpu
def test_a_tokens_bytes_do_not_depend_on_the_batch(api):
    """Alone, in a small call (one chunk a thread) and in a large one (four)."""
    for kv in KV:
        big = Case(api, n=700, kv=kv, heads=(32, 8, 128), rope=(128, 0, False), B=6, seed=2)
        qb = big.run(api)
        want = [t.clone() for t in big.caches]
        for pick in ([5], [640, 17, 5, 699]):
            for t, b in zip(big.caches, big.before):
                t.copy_(b)
            idx = torch.tensor(pick, device="cuda")
            q = api.append(big.prob, big.rope, big.k_new[idx], big.v_new[idx], big.k, big.v,
                           big.i32(big.pos)[idx], rows=big.i32(big.rows)[idx],
                           table=big.i32(big.table), q_new=big.q[idx])
            assert torch.equal(q, qb[idx])
            H, D = big.heads[1:]
            for got, ref in zip(big.caches, want):
                size = {"bf16": 2 * H * D, "e4m3": H * D, "nvfp4": H * D // 2}[kv]
                e = big.entry[pick].cuda()
                cut = big.total * size
                assert torch.equal(got[:cut].view(-1, size)[e], ref[:cut].view(-1, size)[e])
                if kv == "nvfp4":
                    assert torch.equal(got[cut:].view(-1, H * D // 16)[e],
                                       ref[cut:].view(-1, H * D // 16)[e])


@gpu
def test_other_stream_and_graph(api):
    c = Case(api, n=40, kv="e4m3", rope=(128, 0, False), seed=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = c.run(api, stream=side)
    side.synchronize()
    c.check_q(q)
    c.check_caches()
    q0, want = q.clone(), c.caches[0].clone()
    rows, pos, table = c.i32(c.rows), c.i32(c.pos), c.i32(c.table)
    call = lambda: api.append(c.prob, c.rope, c.k_new, c.v_new, c.k, c.v, pos, rows=rows,  # noqa: E731
                              table=table, q_new=c.q, q_out=q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        for t, b in zip(c.caches, c.before):
            t.copy_(b)
        q.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, q0) and torch.equal(c.caches[0], want)


@gpu
def test_a_rotation_described_by_hand(api):
    # da_rope is plain data: filled in field by field it does what rope() gives
    prob = api.problem(batch=3, num_q_heads=4, num_kv_heads=2, head_dim_qk=64, layout="contiguous",
                       scale=0.1, width=8)
    k_new = torch.randn((3, 2, 64), device="cuda")
    freq = torch.rand(32, device="cuda")
    at = torch.tensor([5, 0, 7], dtype=torch.int32, device="cuda")
    got = []
    for rope in (api.rope(freq), api.DaRope(64, 0, 0, 1.0, freq.data_ptr())):
        k, v = (torch.zeros((3, 8, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        api.append(prob, rope, k_new, k_new, k, v, at)
        got.append((k, v))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert got[0][0].any()


@gpu
def test_no_tokens(api):
    c = Case(api, n=3, rope=(128, 0, False))
    q = api.append(c.prob, c.rope, c.k_new[:0], c.v_new[:0], c.k, c.v, c.i32(c.pos)[:0],
                   rows=c.i32(c.rows)[:0], table=c.i32(c.table), q_new=c.q[:0])
    assert q.shape == (0, 8, 128)
    assert all(torch.equal(a, b) for a, b in zip(c.caches, c.before))


# ------------------------------------------------------------------ refusals (no GPU)

def _args(api, **kw):
    fake = 1 << 20  # never dereferenced: every case fails before any device work
    a = dict(n_tokens=4, x_dtype=api.X_BF16, k_new=fake, v_new=fake, q_new=fake, k_stride=1536,
             v_stride=1536, q_stride=1536, positions=fake, rows=fake, table=fake, k=fake, v=fake,
             q_out=1 << 30, err=fake)
    a.update(kw)
    return api.DaAppend(**a)


def _append(api, *structs):
    at = [None if t is None else ctypes.addressof(t) for t in structs]
    return api.lib().decode_attn_append(*at, None)


def _rope(api, **kw):
    r = dict(dim=128, offset=0, interleaved=0, gain=1.0, inv_freq=1 << 20)
    r.update(kw)
    return api.DaRope(**r)


def _prob(api, **kw):
    p = dict(batch=4, num_q_heads=8, num_kv_heads=2, head_dim_qk=128, layout="paged", scale=0.1,
             page_size=16, width=8, num_blocks=40)
    p.update(kw)
    return api.problem(**p)


def test_argument_rules(api):
    def call(prob=None, rope=None, **kw):
        return _append(api, prob or _prob(api), rope or _rope(api), _args(api, **kw))
    bad = api.ERR_INVALID_ARG
    fake = 1 << 20
    assert call(n_tokens=-1) == bad
    assert call(n_tokens=0, k_new=None, v_new=None, k=None) == api.OK
    assert call(x_dtype=2) == bad
    for name in ("k_new", "v_new", "k", "v", "positions", "q_out", "q_new", "table"):
        assert call(**{name: None}) == bad, name
    for name in ("k_new", "v_new", "k", "v", "q_out", "q_new"):
        assert call(**{name: fake + 8}) == bad, name
    for name in ("positions", "rows", "table", "err"):
        assert call(**{name: fake + 2}) == bad, name
    assert call(k_stride=255) == bad and call(v_stride=248) == bad and call(q_stride=1020) == bad
    assert call(k_stride=1537) == bad                      # not a multiple of 16 bytes
    assert call(k_stride=1 << 41) == bad
    assert call(rows=None, n_tokens=5) == bad              # more tokens than rows
    assert call(q_out=fake) == bad                         # over its input
    assert call(q_out=fake + 2 * (3 * 1536 + 512)) == bad  # the input's last 1024 bytes
    for name in ("k_new", "v_new"):                        # over the other inputs
        assert call(**{name: (1 << 30) + 4096}) == bad, name
    for r in (dict(dim=8), dict(dim=-16), dict(offset=4), dict(offset=-8), dict(offset=8),
              dict(dim=144), dict(interleaved=2), dict(gain=float("nan")), dict(inv_freq=None),
              dict(inv_freq=fake + 1)):
        assert call(rope=_rope(api, **r)) == bad, r
    assert call(prob=_prob(api, layout="indexed"), rows=None) == bad
    assert call(prob=_prob(api, page_size=0)) == bad
    latent = dict(num_kv_heads=1, num_q_heads=16, head_dim_qk=576, head_dim_v=512,
                  shared_latent=True, layout="indexed")
    assert call(prob=_prob(api, **latent)) == bad          # a latent cache has no values
    assert call(prob=_prob(api, head_dim_qk=96), rope=_rope(api, dim=64)) == api.ERR_UNSUPPORTED
    assert call(prob=_prob(api, **latent, kv_dtype=api.KV_NVFP4)) == api.ERR_UNSUPPORTED
    assert _append(api, None, None, _args(api)) == bad
    assert _append(api, _prob(api), None, None) == bad


def test_packed_descriptors_match_the_structures(api):
    for packed, c in ((api._APPEND, api.DaAppend), (api._LOGITS, api.Nvfp4Logits)):
        values = list(range(1, len(c._fields_) + 1))
        data = packed.pack(*values)
        assert len(data) == ctypes.sizeof(c)
        s = c.from_buffer_copy(data)
        assert [getattr(s, f[0]) for f in c._fields_] == values


def test_python_refusals(api):
    prob = _prob(api)
    n = 2
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    k = t(40, 16, 2, 128)
    ok = dict(k_new=t(n, 2, 128), v_new=t(n, 2, 128), k=k, v=k,
              positions=t(n, dtype=torch.int32), table=t(4, 8, dtype=torch.int32))

    def refused(match, prob=prob, rope=None, **kw):
        a = {**ok, **kw}
        with pytest.raises(ValueError, match=match):
            api.append(prob, rope, a.pop("k_new"), a.pop("v_new"), a.pop("k"), a.pop("v"),
                       a.pop("positions"), **a)
    refused("CUDA device")  # nothing wrong but the place
    refused("float32 or bfloat16", k_new=t(n, 2, 128, dtype=torch.float16))
    refused("v_new", v_new=t(n, 2, 128, dtype=torch.float32))
    refused("shape", k_new=t(n, 2, 64))
    refused("lie together", k_new=t(n, 128, 2).transpose(1, 2))
    refused("strides", k_new=t(n, 128, 2).transpose(1, 2))
    refused("element type", k=t(40, 16, 2, 128, dtype=torch.uint8))
    refused("holds", k=t(39, 16, 2, 128))
    refused("contiguous", k=t(80, 16, 2, 128)[::2])
    refused("positions", positions=t(n))
    refused("positions", positions=t(n + 1, dtype=torch.int32))
    refused("table", table=None)
    refused("table", table=t(4, 7, dtype=torch.int32))
    refused("v_new and v", v_new=None)
    refused("q_out without", q_out=t(n, 8, 128))
    refused("q_out", q_new=t(n, 8, 128), q_out=t(n, 8, 128, dtype=torch.float32))
    nv = _prob(api, kv_dtype=api.KV_NVFP4)
    refused("holds", prob=nv, k=torch.zeros(40 * 16 * 2 * 64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="inv_freq"):
        api.rope(t(4, 4, dtype=torch.float32))
    with pytest.raises(ValueError, match="inv_freq"):
        api.rope(t(4))


# ------------------------------------------------------------------ the oracle's own pins

def test_oracle_rotation_and_storage():
    x = np.zeros((1, 1, 4))
    x[0, 0] = [1, 2, 3, 4]
    quarter = np.array([np.pi / 2, 0.0], dtype=np.float32)
    np.testing.assert_allclose(OS.rotate(x, [1], quarter)[0, 0], [-3, 2, 1, 4], atol=1e-6)
    np.testing.assert_allclose(OS.rotate(x, [1], quarter, interleaved=True)[0, 0], [-2, 1, 3, 4],
                               atol=1e-6)
    np.testing.assert_allclose(OS.rotate(x, [1], quarter[:1], offset=2, gain=2.0)[0, 0],
                               [1, 2, -8, 6], atol=1e-6)
    v = torch.randn(4000, generator=torch.Generator().manual_seed(1)) * torch.exp2(
        torch.linspace(-14, 9, 4000))
    want = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(OS.store_e4m3(v.double().numpy()), want)
    codes, s = OS.store_nvfp4(np.array([[0, 0.5, -6, 2.5, 5, 0.25, 0.75, 1.25] + [0] * 8]), 1.0)
    assert OF.decode_e4m3(s) == 1.0
    assert ON.decode_e2m1(ON.unpack(codes))[0, :8].tolist() == [0, 0.5, -6, 2, 4, 0, 1, 1]
