"""The operators of a decode step together, as a server runs them: projection,
adapters, rotated append, attention, projection, vocabulary projection, logits.

Every stage is batch-invariant, so a row's whole trajectory -- caches, attention
output, logits and tokens, over several steps -- has the bits of that row run
alone.  The attention of each step is checked against the fp64 oracle on the
cache that the appends have left, and the step captured into a CUDA graph and
replayed gives the eager run's bits."""

import numpy as np
import pytest
import torch

from invariant_decode_attention_gb300 import workloads as W
from oracle import attention as A
from oracle import fp8 as OF
from oracle import nvfp4 as ON
from oracle import step as OS

pytestmark = pytest.mark.gpu

H_Q, H_KV, D, HIDDEN, VOCAB, PAGE, WIDTH = 4, 2, 64, 256, 384, 16, 6
QKV = (H_Q + 2 * H_KV) * D
PROMPTS = [1, 17, 40, 3, 64]
STEPS = 3


@pytest.fixture(scope="module")
def api():
    from invariant_decode_attention_gb300 import api as _api
    _api.lib()
    return _api


class Server:
    """Weights shared by every row, and the state of the rows `who`."""

    def __init__(self, api, who, kv):
        self.api, self.who, B = api, who, len(who)
        dev = "cuda"
        w = lambda N, K, seed: [t.to(dev) if torch.is_tensor(t) else t  # noqa: E731
                                for t in W.nvfp4_weight(N, K, seed, 1.0 / 512)]
        self.w_qkv, self.w_out, self.w_vocab = w(QKV, HIDDEN, 1), w(HIDDEN, H_Q * D, 2), w(VOCAB, HIDDEN, 3)
        g = torch.Generator().manual_seed(4)
        ad = lambda N, K: api.Adapters(  # noqa: E731
            (torch.randn((3, 16, K), generator=g) * K ** -0.5).to(torch.bfloat16).to(dev),
            (torch.randn((3, N, 16), generator=g) * 0.3).to(torch.bfloat16).to(dev),
            torch.tensor([16, 7, 3], dtype=torch.int32, device=dev))
        self.ad_qkv, self.ad_out = ad(QKV, HIDDEN), ad(HIDDEN, H_Q * D)
        self.embed = torch.randn((VOCAB, HIDDEN), generator=g).to(dev)
        self.rope = api.rope((10000.0 ** (-torch.arange(D // 2).double() * 2 / D)).float().to(dev))
        i32 = dict(dtype=torch.int32, device=dev)
        self.ids = torch.tensor([b % 4 - 1 for b in who], **i32)
        pages = B * WIDTH + 2
        perm = np.random.RandomState(B).permutation(pages)[:B * WIDTH].reshape(B, WIDTH)
        self.table = torch.tensor(perm, **i32)
        self.prob = api.problem(batch=B, num_q_heads=H_Q, num_kv_heads=H_KV, head_dim_qk=D,
                                layout="paged", scale=D ** -0.5, page_size=PAGE, width=WIDTH,
                                num_blocks=pages, kv_dtype=kv, k_scale=1 / 32, v_scale=1 / 32)
        shape = (pages, PAGE, H_KV, D)
        if kv == api.KV_BF16:
            self.k, self.v = (torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
        else:
            self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device=dev) for _ in range(2))
        self.kv, self.ws = kv, api.workspace(self.prob)
        self.lengths = torch.zeros(B, **i32)
        self.output = torch.zeros((B, STEPS + 2), **i32)
        self.made = torch.zeros(B, **i32)
        self.prompt = torch.zeros((B, max(PROMPTS)), **i32)
        rows, pos, toks = [], [], []
        for i, b in enumerate(who):
            t = np.random.RandomState(100 + b).randint(0, VOCAB, PROMPTS[b])
            self.prompt[i, :len(t)] = torch.tensor(t)
            rows += [i] * len(t)
            pos += range(len(t))
            toks += list(t)
        self.prompt_lens = torch.tensor([PROMPTS[b] for b in who], **i32)
        rows, pos = torch.tensor(rows + [-1] * 3, **i32), torch.tensor(pos + [0] * 3, **i32)
        x = self.embed[torch.tensor(toks + [0] * 3, device=dev)]  # three padded tokens
        qkv = self.project(x, torch.where(rows >= 0, self.ids[rows.long()], -1).int())
        self.append(qkv, pos, rows)
        self.lengths += self.prompt_lens
        self.token = torch.tensor([toks[int(n) - 1] for n in np.cumsum([PROMPTS[b] for b in who])], **i32)

    def project(self, x, ids):
        y = self.api.nvfp4_mm(x, *self.w_qkv)
        return self.api.nvfp4_adapters(x, self.ad_qkv, ids, y)

    def append(self, qkv, pos, rows=None):
        n = qkv.shape[0]
        cut = [H_Q * D, (H_Q + H_KV) * D]
        return self.api.append(self.prob, self.rope, qkv[:, cut[0]:cut[1]].view(n, H_KV, D),
                               qkv[:, cut[1]:].view(n, H_KV, D), self.k, self.v, pos, rows=rows,
                               table=self.table, q_new=qkv[:, :cut[0]].view(n, H_Q, D))

    def step(self):
        """One token of every row; advances the state on the device."""
        api, B = self.api, len(self.who)
        x = self.embed[self.token.long()]
        q = self.append(self.project(x, self.ids), self.lengths)
        self.lengths += 1
        out = torch.empty((B, H_Q, D), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((B, H_Q), device="cuda")
        api.forward(self.prob, api.INVARIANT, q, self.k, self.v, self.table, self.lengths, self.ws, out,
                    lse)
        attn = out.view(B, H_Q * D)
        o = api.nvfp4_adapters(attn, self.ad_out, self.ids, api.nvfp4_mm(attn, *self.w_out))
        logits = api.nvfp4_mm(x + o, *self.w_vocab)
        self.token = api.nvfp4_logits(
            logits, prompt=self.prompt, prompt_lens=self.prompt_lens, output=self.output,
            output_lens=self.made, repetition=torch.full((B,), 1.3, device="cuda"),
            frequency=torch.full((B,), 0.2, device="cuda"),
            presence=torch.full((B,), 0.1, device="cuda"), out=logits, tokens=self.token)
        self.output.scatter_(1, self.made.long()[:, None], self.token[:, None])
        self.made += 1
        return q, out, lse, logits

    def cache(self, t):
        f = t.float() if self.kv == self.api.KV_BF16 else t.view(torch.float8_e4m3fn).float() / 32
        return f.double().cpu().numpy()


@pytest.mark.parametrize("kv", [0, 1])
def test_rows_alone_and_together(api, kv):
    s = Server(api, list(range(5)), kv)
    solo = [Server(api, [b], kv) for b in range(5)]
    tokens = []
    for _ in range(STEPS):
        got = s.step()
        q, out, lse, logits = got
        ref, ref_lse = A.attend(q.double().cpu().numpy(), s.cache(s.k), s.cache(s.v),
                                s.lengths.cpu().numpy(), scale=D ** -0.5, layout="paged",
                                table=s.table.cpu().numpy(), page_size=PAGE, d_v=D)
        assert np.all(np.abs(out.double().cpu().numpy() - ref) <= np.maximum(1e-2, 2.0 ** -8 * np.abs(ref)))
        assert np.all(np.abs(lse.double().cpu().numpy() - ref_lse) <= 1e-4)
        assert s.token.tolist() == [OS.greedy(r) for r in logits.cpu().numpy()]
        for b, one in enumerate(solo):
            for a, t in zip(got, one.step()):
                assert torch.equal(a[b], t[0]), b
            assert int(one.token) == int(s.token[b])
        tokens.append(s.token.tolist())
    for b, one in enumerate(solo):  # the same entries in other pages
        for mine, theirs in ((s.k, one.k), (s.v, one.v)):
            assert torch.equal(mine[s.table[b].long()], theirs[one.table[0].long()])


def test_a_captured_step_replays(api):
    eager, s = Server(api, [0, 2, 4], 0), Server(api, [0, 2, 4], 0)
    want = [[t.clone() for t in (*eager.step(), eager.token)] for _ in range(STEPS)]
    state = ("k", "v", "lengths", "output", "made", "token")
    saved = {n: getattr(s, n).clone() for n in state}
    keep = {n: getattr(s, n) for n in state}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step()
    torch.cuda.current_stream().wait_stream(side)
    for n in state:
        keep[n].copy_(saved[n])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.step()
    for i in range(STEPS):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*got, s.token), want[i]):
            assert torch.equal(a, b), i


def test_nvfp4_caches_alone_and_together(api):
    """The same over NVFP4 caches: codes of all entries, then their block scales, in
    one buffer."""
    s = Server(api, list(range(5)), api.KV_NVFP4)
    solo = [Server(api, [b], api.KV_NVFP4) for b in range(5)]

    def parts(server, t):
        m, flat = server.prob.num_blocks * PAGE * H_KV * D, t.view(-1)
        return (flat[:m // 2].view(-1, PAGE, H_KV, D // 2),
                flat[m // 2:m // 2 + m // 16].view(-1, PAGE, H_KV, D // 16))

    def values(t):
        codes, scales = parts(s, t)
        step = OF.decode_e4m3(scales.cpu().numpy()) / 32
        return ON.decode_e2m1(ON.unpack(codes.cpu().numpy())) * np.repeat(step, 16, -1)
    for _ in range(STEPS):
        got = s.step()
        ref, ref_lse = A.attend(got[0].double().cpu().numpy(), values(s.k), values(s.v),
                                s.lengths.cpu().numpy(), scale=D ** -0.5, layout="paged",
                                table=s.table.cpu().numpy(), page_size=PAGE, d_v=D)
        out = got[1].double().cpu().numpy()
        assert np.all(np.abs(out - ref) <= np.maximum(1e-2, 2.0 ** -8 * np.abs(ref)))
        assert np.all(np.abs(got[2].double().cpu().numpy() - ref_lse) <= 1e-4)
        assert np.abs(out).max() > 0.1
        for b, one in enumerate(solo):
            for a, t in zip(got, one.step()):
                assert torch.equal(a[b], t[0]), b
    for b, one in enumerate(solo):  # the same entries in other pages
        for mine, theirs in ((s.k, one.k), (s.v, one.v)):
            for x, y in zip(parts(s, mine), parts(one, theirs)):
                assert torch.equal(x[s.table[b].long()], y[one.table[0].long()])
