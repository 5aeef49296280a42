"""nvfp4_mm_logits: penalties, biases and masks on logits and the greedy token.

The library states each step as one fp32 operation, so its logits equal the same
operations in numpy's fp32 bit for bit.  Against fp64 each of the five
operations is off by at most 2^-24 of its result; with R the largest magnitude
on the way (x times or over the repetition penalty, frequency times count, the
bias), the sum is within 6 * 2^-24 * R."""

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
    """Random rows with ragged lists; some lists empty, some tokens repeated."""

    def __init__(self, B, V, *, x="fp32", prompt=40, output=30, bias=6, masks=3, seed=0, pad=0,
                 repeat_bias=False):
        rs = np.random.RandomState(seed)
        self.B, self.V = B, V
        dt = torch.float32 if x == "fp32" else torch.bfloat16
        self.x = torch.from_numpy(rs.standard_normal((B, V + pad)).astype(np.float32) * 3).to(dt)[:, :V]
        tok = lambda w: (rs.random_sample((B, w)) ** 3 * V).astype(np.int32)  # noqa: E731
        self.lists = {}
        for name, w in (("prompt", prompt), ("output", output), ("bias", bias)):
            if not w:
                self.lists[name] = (None, None)
                continue
            lens = rs.randint(0, w + 1, B).astype(np.int32)
            lens[0], lens[-1] = w, 0 if B > 1 else w
            t = tok(w)
            if name == "bias" and not repeat_bias:
                t = np.stack([rs.permutation(max(V, w))[:w] % V for _ in range(B)]).astype(np.int32)
            past = np.arange(w)[None] >= lens[:, None]
            t[past] = 2 ** 31 - 1  # never read
            self.lists[name] = (t, lens)
        self.values = (rs.standard_normal((B, bias)) * 2).astype(np.float32) if bias else None
        self.rep = (rs.random_sample(B) + 0.75).astype(np.float32)
        self.freq = (rs.random_sample(B) - 0.3).astype(np.float32)
        self.pres = (rs.random_sample(B) - 0.3).astype(np.float32)
        self.mask = self.mask_ids = None
        if masks:
            self.mask = rs.randint(-2 ** 31, 2 ** 31, (masks, -(-V // 32)), dtype=np.int64).astype(np.int32)
            self.mask_ids = rs.randint(-1, masks, B).astype(np.int32)

    def kwargs(self):
        c = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        (p, pl), (o, ol), (b, bl) = (self.lists[k] for k in ("prompt", "output", "bias"))
        return dict(prompt=c(p), prompt_lens=c(pl), output=c(o), output_lens=c(ol), bias_tokens=c(b),
                    bias_lens=c(bl), bias_values=c(self.values), repetition=c(self.rep),
                    frequency=c(self.freq), presence=c(self.pres), mask=c(self.mask),
                    mask_ids=c(self.mask_ids))

    def allowed(self, b):
        if self.mask is None:
            return None
        m = b if self.mask_ids is None else self.mask_ids[b]
        if m < 0:
            return None
        bits = np.unpackbits(self.mask[m].astype("<i4").view(np.uint8), bitorder="little")
        return bits[:self.V] != 0

    def part(self, name, b):
        t, lens = self.lists[name]
        t = [] if t is None else t[b, :lens[b]]
        return [v for v in t if 0 <= v < self.V] if name != "bias" else list(t)

    def row(self, b, dtype):
        bias = self.part("bias", b)
        return OS.adjust_logits(self.x[b].float().numpy(), self.part("prompt", b),
                                self.part("output", b), self.rep[b], self.freq[b], self.pres[b],
                                [(v, self.values[b, i]) for i, v in enumerate(bias) if 0 <= v < self.V],
                                self.allowed(b), dtype)

    def check(self, out, tokens):
        out, tokens = out.cpu().numpy(), tokens.cpu().numpy()
        for b in range(self.B):
            same = self.row(b, np.float32)
            assert np.array_equal(out[b], same, equal_nan=True), b
            assert tokens[b] == OS.greedy(same), b
            exact = self.row(b, np.float64)
            made = np.bincount(np.asarray(self.part("output", b), dtype=np.int64), minlength=self.V)
            x = np.abs(self.x[b].double().numpy())
            big = x * max(self.rep[b], 1 / self.rep[b]) + np.abs(self.freq[b]) * made + np.abs(
                self.pres[b])
            for i, v in enumerate(self.part("bias", b)):
                if 0 <= v < self.V:
                    big[v] += abs(self.values[b, i])
            fin = np.isfinite(exact)
            assert np.array_equal(fin, np.isfinite(out[b]))
            assert np.all(np.abs(out[b][fin] - exact[fin]) <= 6 * 2.0 ** -24 * big[fin])


@gpu
@pytest.mark.parametrize("B,V,x,kw", [
    (1, 1, "fp32", dict(bias=1)), (2, 31, "bf16", dict()), (3, 1000, "fp32", dict(masks=0)),
    (4, 4099, "bf16", dict()), (5, 32000, "fp32", dict(prompt=5000, output=700)),
    (2, 65537, "fp32", dict(bias=300)), (3, 70000, "bf16", dict(prompt=0, bias=0)),
    (1, 200064, "bf16", dict(output=2000)), (300, 700, "fp32", dict(output=0)),
    (7, 513, "fp32", dict(prompt=0, output=0, bias=0)),
    (2, 150001, "fp32", dict(prompt=60000, output=30000)), (1, 9000, "bf16", dict(prompt=40000)),
    (160, 70001, "bf16", dict(prompt=300)),
])
def test_against_oracle(api, B, V, x, kw):
    c = Case(B, V, x=x, seed=B + V, **kw)
    out = torch.full((B, V), 123.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens = api.nvfp4_logits(c.x.cuda(), out=out, err=err, **c.kwargs())
    assert int(err) == 0
    c.check(out, tokens)


@gpu
@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("pad,lead", [(0, 0), (4, 0), (3, 1), (8, 4)])
def test_strides_and_alignment(api, x, pad, lead):
    """Rows apart, rows that start anywhere: the bits are those of packed rows."""
    c = Case(6, 1500, x=x, seed=3)
    store = torch.full((6 * (1500 + pad) + lead + 8,), 9.0, dtype=c.x.dtype, device="cuda")
    xs = store[lead:].as_strided((6, 1500), (1500 + pad, 1), lead)
    xs.copy_(c.x)
    outs = torch.full((6 * (1500 + pad) + lead + 8,), 9.0, device="cuda")
    out = outs.as_strided((6, 1500), (1500 + pad, 1), lead)
    tokens = api.nvfp4_logits(xs, out=out, **c.kwargs())
    c.check(out, tokens)
    touched = torch.zeros_like(outs, dtype=torch.bool)
    touched.as_strided((6, 1500), (1500 + pad, 1), lead).fill_(True)
    assert torch.all(outs[~touched] == 9.0)


@gpu
@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("V,pad,lead,apart", [
    (4099, 0, 0, 0), (10003, 0, 1, 0), (8192, 2, 3, 0), (2046, 1, 2, 0), (70001, 4, 1, 0),
    (5000, 1, 0, 4), (40001, 0, 2, 1), (6145, 0, 3, None), (9, 2, 1, 0)])
def test_rows_that_start_off_a_boundary(api, x, V, pad, lead, apart):
    """Rows at every offset from a 16-byte boundary: x and out with the boundaries at the
    same tokens (out `apart` elements on, a multiple of 4), at others, or no out;
    the tokens before a row's first are nobody's."""
    B = 5
    c = Case(B, V, x=x, seed=V + lead, prompt=200, output=100)
    prompt, lens = c.lists["prompt"]
    prompt[:, :7] = [-1, -2, -3, 0, 1, 2, V]  # three in front of the row, one behind it
    lens[:-1] = np.maximum(lens[:-1], 7)
    size = B * (V + pad) + 64
    store = torch.full((size,), 1e30, dtype=c.x.dtype, device="cuda")  # beats all if it is read
    xs = store.as_strided((B, V), (V + pad, 1), 16 + lead)
    xs.copy_(c.x)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    packed = torch.empty((B, V), device="cuda")
    want = api.nvfp4_logits(c.x.cuda(), out=packed, **c.kwargs())
    if apart is None:
        tokens = api.nvfp4_logits(xs, err=err, **c.kwargs())
    else:
        outs = torch.full((size + 8,), 9.0, device="cuda")
        out = outs.as_strided((B, V), (V + pad, 1), 16 + lead + apart)
        tokens = api.nvfp4_logits(xs, out=out, err=err, **c.kwargs())
        c.check(out, tokens)
        assert torch.equal(out, packed)
        touched = torch.zeros_like(outs, dtype=torch.bool)
        touched.as_strided((B, V), (V + pad, 1), 16 + lead + apart).fill_(True)
        assert torch.all(outs[~touched] == 9.0)
        if x == "fp32" and apart == 0:  # in place
            assert torch.equal(api.nvfp4_logits(xs, out=xs, **c.kwargs()), tokens)
            assert torch.equal(xs, packed)
    assert torch.equal(tokens, want) and int(err) == api.DEVERR_INDEX


@gpu
@pytest.mark.parametrize("x", ["fp32", "bf16"])
def test_rows_of_x_and_out_side_by_side(api, x):
    # one buffer's rows hold both: they interleave and do not overlap
    B, V = 5, 1500
    c = Case(B, V, x=x, seed=6)
    packed = torch.empty((B, V), device="cuda")
    want = api.nvfp4_logits(c.x.cuda(), out=packed, **c.kwargs())
    size = 4 if x == "fp32" else 2
    for x_first in (True, False):
        rows = torch.full((B, V * (size + 4)), 77, dtype=torch.uint8, device="cuda")
        cut = V * (size if x_first else 4)
        xs, out = (rows[:, :cut], rows[:, cut:]) if x_first else (rows[:, cut:], rows[:, :cut])
        xs, out = xs.view(c.x.dtype), out.view(torch.float32)
        xs.copy_(c.x)
        assert torch.equal(api.nvfp4_logits(xs, out=out, **c.kwargs()), want)
        assert torch.equal(out, packed) and torch.equal(xs, c.x.cuda())


@gpu
@pytest.mark.parametrize("B,V", [(2, 1 << 30), (3, (1 << 30) - 1), (17000, 131073)])
def test_offsets_beyond_32_bits(api, B, V):
    """More than 2^31 logits: the largest vocabulary, and many rows."""
    x = torch.zeros((B, V), device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    last = B - 1
    x[0, V - 1], x[0, V - 2], x[last, V - 1], x[last, 5] = 5.0, 4.0, -1.0, 2.0
    prompt = torch.full((B, 1), V - 1, **i32)
    lens = torch.zeros(B, **i32)
    lens[0] = lens[last] = 1
    bias = torch.zeros((B, 1), **i32)
    bias[last] = V - 7
    out = torch.empty_like(x)
    tokens = api.nvfp4_logits(x, prompt=prompt, prompt_lens=lens, out=out, bias_tokens=bias,
                              repetition=torch.full((B,), 2.0, device="cuda"),
                              bias_values=torch.full((B, 1), 3.0, device="cuda"),
                              bias_lens=torch.where(torch.arange(B, device="cuda") == last, 1, 0).int())
    x[0, V - 1], x[last, V - 1], x[last, V - 7] = 2.5, -2.0, 3.0
    assert all(torch.equal(out[b0:b0 + 1000], x[b0:b0 + 1000]) for b0 in range(0, B, 1000))
    want = torch.zeros(B, dtype=torch.int32)
    want[0], want[last] = V - 2, V - 7
    assert torch.equal(tokens.cpu(), want)
    del x, out
    torch.cuda.empty_cache()


@gpu
@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [2, 33, 2049, 6147, 50001])
def test_single_rows_of_any_length(api, x, V):
    # one row takes no notice of a stride: aligned, it moves in groups of four to its last step
    c = Case(1, V, x=x, seed=V, prompt=60, output=50, bias=min(6, V))
    out = torch.full((1, V + 3), 5.0, device="cuda")
    tokens = api.nvfp4_logits(c.x.cuda(), out=out[:, :V], **c.kwargs())
    c.check(out[:, :V], tokens)
    assert torch.all(out[:, V:] == 5.0)
    assert torch.equal(api.nvfp4_logits(c.x.cuda(), **c.kwargs()), tokens)


@gpu
def test_in_place_and_tokens_only(api):
    c = Case(9, 3001, seed=31, repeat_bias=True, bias=40)
    x = c.x.cuda().contiguous()
    only = api.nvfp4_logits(x, **c.kwargs())
    assert torch.equal(x.cpu(), c.x)  # not written
    tokens = api.nvfp4_logits(x, out=x, **c.kwargs())
    c.check(x, tokens)
    assert torch.equal(only, tokens)


@gpu
def test_repeated_bias_tokens_add_up_in_order(api):
    V = 64
    x = torch.zeros((1, V), device="cuda")
    bt = torch.tensor([[5, 7, 5, 5, 7, 9]], dtype=torch.int32, device="cuda")
    bv = torch.tensor([[1e8, 2.0, 1.0, -1e8, 3.0, 0.5]], device="cuda")
    out = torch.empty_like(x)
    api.nvfp4_logits(x, bias_tokens=bt, bias_values=bv, out=out,
                     bias_lens=torch.tensor([5], dtype=torch.int32, device="cuda"))
    want = torch.zeros(V)
    want[5], want[7] = 0.0, 5.0  # (1e8 + 1) - 1e8 = 0 in fp32, in this order; 9 is past the length
    assert torch.equal(out[0].cpu(), want)


@gpu
def test_the_longest_bias_list(api):
    V, W = 9000, api.LOGITS_MAX_BIAS
    g = torch.Generator().manual_seed(3)
    x = torch.randn((2, V), generator=g)
    at = torch.stack([torch.randperm(V, generator=g)[:W] for _ in range(2)]).to(torch.int32)
    v = torch.randn((2, W), generator=g)
    want = x.scatter_add(1, at.long(), v)  # distinct tokens: one addition each
    out = torch.empty((2, V), device="cuda")
    tokens = api.nvfp4_logits(x.cuda(), bias_tokens=at.cuda(), bias_values=v.cuda(), out=out,
                              bias_lens=torch.full((2,), W, dtype=torch.int32, device="cuda"))
    assert torch.equal(out.cpu(), want)
    assert torch.equal(tokens.cpu().long(), want.argmax(1))


@gpu
def test_greedy_ties_masks_infinities_and_nan(api):
    nan, inf = float("nan"), float("inf")
    V = 9000  # several CTAs a row
    x = torch.full((9, V), -5.0, device="cuda")
    x[0, [8000, 70, 4000]] = 2.0          # the lowest of equals
    x[1] = -inf                           # nothing to pick
    x[2, 100], x[2, 50] = nan, 1.0        # a NaN is never picked
    x[3] = nan
    x[4, [8500, 3]] = inf
    x[5, 20], x[5, 10] = 0.0, -0.0        # equal: the lower
    x[6] = torch.finfo(torch.float32).min  # finite, so picked
    words = -(-V // 32)
    mask = torch.full((9, words), -1, dtype=torch.int32, device="cuda")
    mask[7] = 0                           # the mask leaves nothing
    mask[8] = 0
    mask[8, 7000 // 32] = 1 << (7000 % 32)
    x[8, 7000] = -1e30
    out = torch.empty_like(x)
    tokens = api.nvfp4_logits(x, mask=mask, out=out)
    assert tokens.tolist() == [70, -1, 50, -1, 3, 10, 0, -1, 7000]
    assert torch.all(out[7] == -inf) and int(torch.isfinite(out[8]).sum()) == 1
    # a masked place's own value does not matter
    x[8] = nan
    x[8, 7000] = -1e30
    x[8, 1] = inf
    assert api.nvfp4_logits(x, mask=mask, out=out).tolist()[8] == 7000
    assert int(torch.isnan(out[8]).sum()) == 0


@gpu
@pytest.mark.parametrize("L", [8191, 8192, 70000])
def test_many_repeats_of_one_token(api, L):
    # counts do not spill into each other (L even: half the second row's)
    V = 40
    o = torch.full((2, L), 3, dtype=torch.int32, device="cuda")
    o[1, ::2] = 4
    x = torch.zeros((2, V), device="cuda")
    out = torch.empty_like(x)
    one = torch.ones(2, device="cuda")
    api.nvfp4_logits(x, output=o, output_lens=torch.full((2,), L, dtype=torch.int32, device="cuda"),
                     frequency=one, presence=one, out=out)
    want = torch.zeros(2, V)
    want[0, 3], want[1, 3], want[1, 4] = -L - 1.0, -(L // 2) - 1.0, -((L + 1) // 2) - 1.0
    assert torch.equal(out.cpu(), want)


@gpu
def test_row_bits_do_not_depend_on_the_batch(api):
    c = Case(12, 5000, seed=77)
    kw = c.kwargs()
    x = c.x.cuda()
    out = torch.empty((12, 5000), device="cuda")
    tokens = api.nvfp4_logits(x, out=out, **kw)
    for pick in ([3], [11, 0, 7], list(range(11, -1, -1))):
        sub = {k: (v if v is None or k == "mask" else v[pick].contiguous()) for k, v in kw.items()}
        o = torch.empty((len(pick), 5000), device="cuda")
        t = api.nvfp4_logits(x[pick], out=o, **sub)
        assert torch.equal(o, out[pick]) and torch.equal(t, tokens[pick])


@gpu
def test_bad_entries_are_skipped_and_flagged(api):
    c = Case(4, 300, seed=5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty((4, 300), device="cuda")

    def run():
        err.zero_()
        return api.nvfp4_logits(c.x.cuda(), out=out, err=err, **c.kwargs())
    for name in ("prompt", "output", "bias"):
        t, lens = c.lists[name]
        for bad in (-1, 300, -2 ** 31, 2 ** 31 - 1):
            keep = t[0, 2]
            t[0, 2] = bad
            tokens = run()
            assert int(err) == api.DEVERR_INDEX, (name, bad)
            c.check(out, tokens)
            t[0, 2] = keep
        w = t.shape[1]
        for bad, used in ((w + 1, w), (2 ** 31 - 1, w), (-1, 0)):
            t[3, :] = np.arange(w)
            keep, lens[3] = lens[3], bad
            tokens = run()
            assert int(err) == api.DEVERR_LENGTH, (name, bad)
            lens[3] = used
            c.check(out, tokens)
            lens[3] = keep
    c.mask_ids[1] = 3
    tokens = run()
    assert int(err) == api.DEVERR_INDEX
    c.mask_ids[1] = -1
    c.check(out, tokens)
    api.nvfp4_logits(c.x.cuda(), out=out, **c.kwargs())  # no error word: nothing to set


@gpu
def test_repeats_stream_and_graph(api):
    c = Case(20, 9001, seed=41)
    kw, x = c.kwargs(), c.x.cuda()
    out, tokens = torch.empty((20, 9001), device="cuda"), torch.empty(20, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    api.nvfp4_logits(x, out=out, tokens=tokens, stream=side, **kw)
    side.synchronize()
    c.check(out, tokens)
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.nvfp4_logits(x, out=out, tokens=tokens, **kw)
    for _ in range(3):
        out.zero_(), tokens.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        c.check(out, tokens)


@gpu
def test_no_rows_and_empty_lists(api):
    x = torch.randn((3, 100), device="cuda")
    assert api.nvfp4_logits(x[:0]).shape == (0,)
    none = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    t = api.nvfp4_logits(x, prompt=none, prompt_lens=lens, output=none, output_lens=lens,
                         bias_tokens=none, bias_values=none.float(), bias_lens=lens, out=out)
    assert torch.equal(out, x) and torch.equal(t.long(), x.argmax(-1))


# ------------------------------------------------------------------ refusals (no GPU)

def test_argument_rules(api):
    fake = 1 << 20  # never dereferenced: every case fails before any device work

    def call(**kw):
        a = dict(batch=2, vocab=1000, x_dtype=api.X_F32, x=fake, x_stride=1000, out=1 << 28,
                 out_stride=1000, tokens=fake)
        a.update(kw)
        g = api.Nvfp4Logits(**a)
        return api.lib().nvfp4_mm_logits(ctypes.addressof(g), None)
    bad = api.ERR_INVALID_ARG
    assert api.lib().nvfp4_mm_logits(None, None) == bad
    assert call(batch=-1) == bad and call(vocab=0) == bad and call(x_dtype=5) == bad
    assert call(vocab=(1 << 30) + 1) == api.ERR_UNSUPPORTED
    assert call(batch=0, x=None, out=None, tokens=None) == api.OK
    assert call(x=None) == bad and call(x_stride=999) == bad and call(x=fake + 2) == bad
    assert call(out=None, tokens=None) == bad and call(out_stride=999) == bad
    assert call(out=(1 << 28) + 2) == bad
    for name in ("prompt", "output"):
        assert call(**{name: fake, name + "_width": 4}) == bad
        assert call(**{name + "_lens": fake, name + "_width": 4}) == bad
        assert call(**{name: fake, name + "_lens": fake, name + "_width": -1}) == bad
        assert call(**{name: fake + 1, name + "_lens": fake, name + "_width": 4}) == bad
    assert call(bias_tokens=fake, bias_lens=fake, bias_width=3) == bad
    assert call(bias_values=fake, bias_width=3) == bad
    wide = dict(bias_tokens=fake, bias_values=fake, bias_lens=fake)
    assert call(**wide, bias_width=api.LOGITS_MAX_BIAS + 1) == api.ERR_UNSUPPORTED
    wide = dict(prompt=fake, prompt_lens=fake, prompt_width=1 << 28, output=fake, output_lens=fake)
    assert call(**wide, output_width=1 << 28) == api.ERR_UNSUPPORTED
    assert call(mask=fake, n_masks=0, mask_ids=fake) == bad
    assert call(mask=fake, n_masks=1) == bad           # two rows, no ids
    assert call(mask_ids=fake) == bad
    for name in ("repetition", "frequency", "presence", "tokens", "err"):
        assert call(**{name: fake + 2}) == bad, name
    assert call(out=fake + 4000) == bad                # inside x
    assert call(out=fake, out_stride=1004) == bad      # in place, other rows
    assert call(x_dtype=api.X_BF16, out=fake) == bad   # in place, other type


def test_rows_that_interleave_and_overlap(api):
    fake = 1 << 20  # never dereferenced: every case is refused before any device work

    def call(**kw):
        a = dict(batch=3, vocab=1000, x_dtype=api.X_F32, x=fake, x_stride=2500, out_stride=2500,
                 tokens=fake)
        a.update(kw)
        g = api.Nvfp4Logits(**a)
        return api.lib().nvfp4_mm_logits(ctypes.addressof(g), None)
    for at in (4, 999, 1501, 2499, 2500, 2501, 5000, 5999, -4, -999, -2500, -2501, -5999):
        assert call(out=fake + 4 * at) == api.ERR_INVALID_ARG, at
    # bf16 x, rows of the same size: 500 words of x to 1000 of out
    half = dict(x_dtype=api.X_BF16, x_stride=5000)
    for at in (0, 499, 1501, 2500, 2999, -1, -999, -2500, -5999):
        assert call(out=fake + 4 * at, **half) == api.ERR_INVALID_ARG, at
    # rows of two sizes: refused as soon as the two buffers touch
    assert call(out=fake + 4000, out_stride=2504) == api.ERR_INVALID_ARG


def test_strides_without_end(api):
    fake = 1 << 20  # never dereferenced: every case is refused before any device work

    def call(**kw):
        a = dict(batch=3, vocab=1000, x_dtype=api.X_F32, x=fake, x_stride=1000, out=1 << 28,
                 out_stride=1000, tokens=fake)
        a.update(kw)
        g = api.Nvfp4Logits(**a)
        return api.lib().nvfp4_mm_logits(ctypes.addressof(g), None)
    for big in ((1 << 40) + 1, 1 << 61, 1 << 62, (1 << 63) - 1):
        for x_dtype in (api.X_F32, api.X_BF16):
            both = dict(x_stride=big, out_stride=big, x_dtype=x_dtype)
            assert call(**both) == api.ERR_INVALID_ARG
            assert call(**both, out=fake + 64) == api.ERR_INVALID_ARG
            # one row's stride does not matter, but that it overlaps does
            assert call(**both, batch=1, out=fake + 64) == api.ERR_INVALID_ARG
        assert call(x_stride=big) == api.ERR_INVALID_ARG
        assert call(out_stride=big) == api.ERR_INVALID_ARG


def test_python_refusals(api):
    t = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype)  # noqa: E731
    i32 = torch.int32

    def refused(match, x=t(2, 50), **kw):
        with pytest.raises(ValueError, match=match):
            api.nvfp4_logits(x, tokens=kw.pop("tokens", t(2, dtype=i32)), **kw)
    refused("CUDA device")
    refused("float32 or bfloat16", x=t(2, 50, dtype=torch.float16))
    refused("strides", x=t(2, 100)[:, ::2])
    refused("belong together", prompt=t(2, 5, dtype=i32))
    refused("belong together", bias_values=t(2, 5))
    refused("prompt", prompt=t(3, 5, dtype=i32), prompt_lens=t(2, dtype=i32))
    refused("output", output=t(2, 5), output_lens=t(2, dtype=i32))
    refused("output_lens", output=t(2, 5, dtype=i32), output_lens=t(3, dtype=i32))
    refused("bias_values", bias_tokens=t(2, 5, dtype=i32), bias_lens=t(2, dtype=i32),
            bias_values=t(2, 4))
    refused("repetition", repetition=t(3))
    refused("mask", mask=t(1, 2), mask_ids=t(2, dtype=i32))
    refused("mask", mask=t(1, 3, dtype=i32), mask_ids=t(2, dtype=i32))
    refused("out", out=t(2, 51))
    refused("tokens", tokens=t(2))


def test_oracle_on_a_hand_made_row():
    l = OS.adjust_logits([2.0, -2.0, 4.0, 1.0, 0.5], prompt=[0], output=[1, 2, 2], repetition=2.0,
                         frequency=0.25, presence=0.5, bias=[(3, 1.0), (3, 2.0)],
                         allowed=np.array([1, 1, 1, 1, 0], bool))
    assert l.tolist() == [1.0, -4.75, 1.0, 4.0, -np.inf]
    assert OS.greedy(l) == 3
    assert OS.greedy(np.array([-np.inf, np.nan])) == -1
