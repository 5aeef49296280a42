"""Cases, plain forms and exact values of three operators of a decode step:

* append: new keys and values rotated by their positions and written into the
  cache that decode attention reads (queries rotated in the same pass);
* adapters: low-rank adapters of many requests added to the output of a shared
  weight matmul;
* logits: penalties for repeated tokens, biases and grammar masks on the logits
  of the vocabulary projection, and the greedy token.

``listed()`` names the cases that are timed, ``draw(rng)`` gives others of the
same ranges; ``prepare``/``run`` make the inputs and do one pass, in plain
torch operations or (``own``) through the package's entry points.
"""

import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "fp32": F32}


# ------------------------------------------------------------------ cases

def listed():
    gqa = dict(H_q=32, H_kv=8, D=128, rope_dim=128, rope_offset=0, interleaved=False)
    return [
        # one request decodes one token: nothing but latency
        dict(name="append_1", op="append", n=1, seqs=1, context=4096, pad=0, layout="paged", page=16,
             kv="bf16", x="bf16", latent=False, **gqa),
        # a decode step of 32 requests, fp32 projections, E4M3 cache
        dict(name="append_32_e4m3", op="append", n=32, seqs=32, context=2048, pad=0, layout="paged",
             page=16, kv="e4m3", x="fp32", latent=False, **gqa),
        # 64 requests over a shared latent cache of 65536 slots; 64 of 576 dims rotate, in pairs
        dict(name="append_latent_64", op="append", n=64, seqs=64, context=65536, pad=3, layout="indexed",
             page=0, kv="bf16", x="bf16", latent=True, H_q=128, H_kv=1, D=576, rope_dim=64,
             rope_offset=512, interleaved=True),
        # three ragged prompts into an NVFP4 cache, a quarter of each head rotated, padded batch
        dict(name="append_prompt_nvfp4", op="append", n=2047, seqs=3, context=1024, pad=17, layout="paged",
             page=48, kv="nvfp4", x="bf16", latent=False, H_q=32, H_kv=8, D=128, rope_dim=32,
             rope_offset=0, interleaved=False),
        # long prompts: the largest append
        dict(name="append_prompt_bf16", op="append", n=16384, seqs=5, context=6144, pad=0, layout="paged",
             page=64, kv="bf16", x="bf16", latent=False, **gqa),
        # one row, one adapter beside the 4096 -> 8192 projection
        dict(name="adapters_1", op="adapters", n=1, K=4096, N=8192, count=4, rank=16, x="fp32", y="fp32"),
        # a decode step whose rows use 24 adapters of ranks 64, 32 and 16, some rows none
        dict(name="adapters_67", op="adapters", n=67, K=4096, N=8192, count=24, rank=64, x="bf16", y="fp32"),
        # prompts of 8 requests, one adapter each, with the bf16 copy of the result
        dict(name="adapters_prompt", op="adapters", n=8192, K=4096, N=8192, count=8, rank=64, x="bf16",
             y="both"),
        # one request's greedy token, the adjusted logits not wanted
        dict(name="logits_1", op="logits", B=1, V=32000, history=300, biases=4, mask=False, x="fp32",
             write=False),
        # a decode step with an odd vocabulary, everything switched on
        dict(name="logits_33_odd", op="logits", B=33, V=50001, history=3000, biases=40, mask=True, x="bf16",
             write=True),
        # a large step, adjusted logits wanted (a sampler follows)
        dict(name="logits_256", op="logits", B=256, V=131072, history=4000, biases=16, mask=True, x="fp32",
             write=True),
        # long histories against a small vocabulary
        dict(name="logits_64_long", op="logits", B=64, V=32000, history=30000, biases=0, mask=False,
             x="bf16", write=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "adapters", "logits"])
    if op == "append":
        latent = rng.random() < 0.2
        if latent:
            H_q, H_kv, D = rng.choice([16, 64, 128]), 1, 576
            rope = dict(rope_dim=64, rope_offset=512, interleaved=rng.random() < 0.7)
            layout, kv = rng.choice(["paged", "indexed", "contiguous"]), rng.choice(["bf16", "e4m3"])
            most = 1024
        else:
            H_q, H_kv, D = rng.choice([(32, 8, 128), (8, 1, 64), (128, 8, 128), (20, 4, 64), (7, 7, 128),
                                       (48, 2, 128)])
            dim = rng.choice([D, D, D // 2, 32])
            rope = dict(rope_dim=dim, rope_offset=rng.choice([0, D - dim]),
                        interleaved=rng.random() < 0.3)
            layout, kv = rng.choice(["paged", "paged", "indexed", "contiguous"]), rng.choice(
                ["bf16", "e4m3", "nvfp4"])
            most = 16384 * 48 * 128 // ((H_q + 2 * H_kv) * D)
        n = _log(rng, 1, min(most, 16384))
        seqs = n if n <= 256 and rng.random() < 0.6 else rng.randint(1, min(n, 8))
        context = max(_log(rng, 64, 2048), -(-n // seqs) * 2)
        return dict(op=op, n=n, seqs=seqs, context=65536 if layout == "indexed" else context,
                    pad=rng.choice([0, 0, rng.randint(0, n // 8)]), layout=layout,
                    page=rng.choice([1, 16, 48, 64]) if layout == "paged" else 0, kv=kv,
                    x=rng.choice(["bf16", "fp32"]), latent=latent, H_q=H_q, H_kv=H_kv, D=D, **rope)
    if op == "adapters":
        n = _log(rng, 1, 8192)
        K, N = 64 * _log(rng, 4, 128), 128 * _log(rng, 1, 64)
        rank = rng.choice([16, 32, 48, 64, 128])
        count = _log(rng, 1, 64)
        while n * count * rank * (K + N) > 8192 * 8 * 64 * 12288:
            count = max(1, count // 2)
            n = n if count > 1 else n // 2
        return dict(op=op, n=n, K=K, N=N, count=count, rank=rank, x=rng.choice(["bf16", "fp32"]),
                    y=rng.choice(["fp32", "both"]))
    V = _log(rng, 1000, 131072)
    B = _log(rng, 1, 256)
    return dict(op=op, B=B, V=V, history=_log(rng, 1, 30000) if B <= 64 else _log(rng, 1, 4000),
                biases=rng.choice([0, 4, 40, 300]), mask=rng.random() < 0.5, x=rng.choice(["bf16", "fp32"]),
                write=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, g, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32).to(dtype)


def _randint(lo, hi, shape, g):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)


def _ragged(total, parts, rs):
    """`parts` positive lengths with the sum `total`."""
    cuts = np.sort(rs.choice(np.arange(1, total), parts - 1, replace=False)) if parts > 1 else []
    return np.diff(np.concatenate([[0], cuts, [total]]).astype(np.int64))


def prepare(case, seed):
    return {"append": _prepare_append, "adapters": _prepare_adapters,
            "logits": _prepare_logits}[case["op"]](case, seed)


def _prepare_append(c, seed):
    """The projections of n tokens (q, k and v side by side in one row, as a
    fused projection leaves them), the cache with what it already holds, and
    where each token goes.  The last `pad` tokens are padding (row -1)."""
    g, rs = _gen(seed), np.random.RandomState(seed % (1 << 31))
    n, B, H_q, H_kv, D = c["n"], c["seqs"], c["H_q"], c["H_kv"], c["D"]
    x_type = TYPES[c["x"]]
    D_v = 512 if c["latent"] else D
    if c["latent"]:
        q = _randn((n, H_q, D), g, x_type)
        k_new, v_new = _randn((n, 1, D), g, x_type), None
    else:
        qkv = _randn((n, (H_q + 2 * H_kv) * D), g, x_type)
        q = qkv[:, :H_q * D].view(n, H_q, D)
        k_new = qkv[:, H_q * D:(H_q + H_kv) * D].view(n, H_kv, D)
        v_new = qkv[:, (H_q + H_kv) * D:].view(n, H_kv, D)

    live = n - c["pad"]
    if B == n:  # decode: one token a row, anywhere in its context
        start, new = rs.randint(0, c["context"], B), np.ones(B, np.int64)
    else:       # prompts: a run of new tokens after what the row already has
        new = _ragged(n, B, rs)
        start = np.array([rs.randint(0, max(1, c["context"] - m + 1)) for m in new])
    rows = np.repeat(np.arange(B), new)
    positions = np.concatenate([np.arange(s, s + m) for s, m in zip(start, new)])
    longest = max(c["context"], n - B + 1)  # a row's room, the same for every seed
    table, page = None, max(c["page"], 1)
    if c["layout"] == "paged":
        need = -(-(start + new) // page)
        width = -(-longest // page)
        pages = B * width + 3
        order = rs.permutation(pages)[:int(need.sum())]
        tab = np.full((B, width), -1, np.int64)
        for b, (m, at) in enumerate(zip(need, np.cumsum(need) - need)):
            tab[b, :m] = order[at:at + m]
        lead, entry = (pages, page), tab[rows, positions // page] * page + positions % page
        table = torch.tensor(tab, dtype=torch.int32, device="cuda")
    elif c["layout"] == "contiguous":
        width = longest
        lead, entry = (B, width), rows * width + positions
    else:  # one slot a token, any free one
        width = 0
        lead, entry = (c["context"],), rs.permutation(c["context"])[:n]
        rows = entry
    rows = np.where(np.arange(n) < live, rows, -1)

    kv = {}
    total = int(np.prod(lead))
    for name, dim in (("k", D), ("v", D)):
        if name == "v" and c["latent"]:
            kv["v"] = None
        elif c["kv"] == "bf16":
            kv[name] = _randn((*lead, H_kv, dim), g, BF16)
        elif c["kv"] == "e4m3":
            kv[name] = (_randn((*lead, H_kv, dim), g) * 16).to(torch.float8_e4m3fn)
        else:  # codes of all entries, then their block scales, in one buffer
            m = total * H_kv * dim
            kv[name] = torch.empty(m // 2 + m // 16, dtype=torch.uint8, device="cuda")
            kv[name][:m // 2] = _randint(0, 256, (m // 2,), g).to(torch.uint8)
            kv[name][m // 2:] = _randint(32, 64, (m // 16,), g).to(torch.uint8)
    half = c["rope_dim"] // 2
    inv_freq = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(case=c, q=q, k_new=k_new, v_new=v_new, inv_freq=inv_freq, live=live, total=total,
             q_out=torch.zeros((n, H_q, D), dtype=BF16, device="cuda"),
             positions=torch.tensor(positions, **i32), rows=torch.tensor(rows, **i32), table=table,
             entry=torch.tensor(entry[:live], device="cuda"), k_scale=1.0 / 64, v_scale=1.0 / 48,
             e2m1_bytes=_e2m1_bytes() if c["kv"] == "nvfp4" else None, **kv)
    if own:  # what a server makes once: the problem's description and the rotation's
        from invariant_decode_attention_gb300 import api
        s["prob"] = api.problem(batch=B, num_q_heads=H_q, num_kv_heads=H_kv, head_dim_qk=D, head_dim_v=D_v,
                                layout=c["layout"], scale=D ** -0.5, page_size=c["page"], width=max(width, 1),
                                num_blocks=lead[0] if c["layout"] != "contiguous" else 0,
                                shared_latent=c["latent"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                kv_dtype={"bf16": api.KV_BF16, "e4m3": api.KV_FP8_E4M3,
                                          "nvfp4": api.KV_NVFP4}[c["kv"]])
        s["rope"] = api.rope(inv_freq, offset=c["rope_offset"], interleaved=c["interleaved"])
    return s


def _ranks(c):
    """An adapter's rank: the full one, a half or a quarter, in turn."""
    return [max(1, c["rank"] >> (a % 3)) for a in range(c["count"])]


def _adapter_of(c):
    """Which adapter each row uses: the same number of rows for each, every
    (count + 1)-th share of a decode step none (-1); prompts' rows in runs."""
    ids = np.arange(c["n"]) % (c["count"] + 1)
    ids[ids == c["count"]] = -1
    return np.sort(ids) if c["n"] > 512 else ids


def _prepare_adapters(c, seed):
    g, rs = _gen(seed), np.random.RandomState(seed % (1 << 31))
    n, K, N, count, rank = (c[k] for k in ("n", "K", "N", "count", "rank"))
    ids = _adapter_of(c)
    if c["n"] <= 512:
        ids = ids[rs.permutation(n)]
    s = dict(case=c, x=_randn((n, K), g, TYPES[c["x"]]), y=_randn((n, N), g),
             a=(_randn((count, rank, K), g) * K ** -0.5).to(BF16),
             b=(_randn((count, N, rank), g) * 0.1).to(BF16),
             ranks=torch.tensor(_ranks(c), dtype=torch.int32, device="cuda"),
             scales=torch.rand(count, generator=g, device="cuda") + 0.5,
             ids=torch.tensor(ids, dtype=torch.int32, device="cuda"),
             out=torch.zeros((n, N), device="cuda"),
             out_bf16=torch.zeros((n, N), dtype=BF16, device="cuda") if c["y"] == "both" else None)
    if own:  # what a server makes once: the adapters' handle and the workspace
        from invariant_decode_attention_gb300 import api
        s["handle"] = api.Adapters(s["a"], s["b"], s["ranks"], s["scales"])
        s["ws"] = api.adapters_workspace(n, N, K, s["handle"])
    return s


def _lengths(B, most, rs):
    return np.minimum(most, np.maximum(0, (most * rs.random_sample(B) * 1.2).astype(np.int64)))


def _prepare_logits(c, seed):
    """Logits of a vocabulary projection; each row's prompt and output tokens
    (few distinct ones often: drawn with a power), padded to the longest."""
    g, rs = _gen(seed), np.random.RandomState(seed % (1 << 31))
    B, V, L, W = c["B"], c["V"], c["history"], c["biases"]
    i32 = dict(dtype=torch.int32, device="cuda")

    def tokens(width):
        u = torch.rand((B, width), generator=g, device="cuda")
        return (u.pow(4) * V).to(torch.int32).clamp_(max=V - 1)

    p_most, o_most = max(1, L - L // 3), max(1, L // 3)
    s = dict(case=c, x=_randn((B, V), g, TYPES[c["x"]]) * 3,
             prompt=tokens(p_most), prompt_lens=torch.tensor(_lengths(B, p_most, rs), **i32),
             output=tokens(o_most), output_lens=torch.tensor(_lengths(B, o_most, rs), **i32),
             repetition=torch.rand(B, generator=g, device="cuda") + 0.75,
             frequency=torch.rand(B, generator=g, device="cuda") - 0.25,
             presence=torch.rand(B, generator=g, device="cuda") - 0.25,
             bias_tokens=None, bias_values=None, bias_lens=None, mask=None, mask_ids=None,
             out=torch.zeros((B, V), device="cuda") if c["write"] else None,
             tokens=torch.zeros(B, **i32))
    if W:
        W = min(W, V)
        start = torch.tensor(rs.randint(0, V, (B, 1)), device="cuda")
        s["bias_tokens"] = ((start + torch.arange(W, device="cuda") * max(1, V // W)) % V).to(torch.int32)
        s["bias_values"] = _randn((B, W), g) * 2
        s["bias_lens"] = torch.tensor(_lengths(B, W, rs), **i32)
    if c["mask"]:  # a few grammars' masks, shared by rows; a bit for each token; -1: any token
        words = -(-V // 32)
        s["mask"] = _randint(-2 ** 31, 2 ** 31 - 1, (4, words), g) & _randint(-2 ** 31, 2 ** 31 - 1, (4, words), g)
        s["mask_ids"] = torch.tensor(rs.randint(-1, 4, B), **i32)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return {"append": _own_append, "adapters": _own_adapters, "logits": _own_logits}[s["case"]["op"]](s)
    return {"append": _plain_append, "adapters": _plain_adapters, "logits": _plain_logits}[s["case"]["op"]](s)


def _own_append(s):
    from invariant_decode_attention_gb300 import api
    api.append(s["prob"], s["rope"], s["k_new"], s["v_new"], s["k"], s["v"], s["positions"], rows=s["rows"],
               table=s["table"], q_new=s["q"], q_out=s["q_out"])
    return _append_outputs(s)


def _own_adapters(s):
    from invariant_decode_attention_gb300 import api
    api.nvfp4_adapters(s["x"], s["handle"], s["ids"], s["y"], out=s["out"], out_bf16=s["out_bf16"], ws=s["ws"])
    return {"y": s["out"], "y_bf16": s["out_bf16"]}


def _own_logits(s):
    from invariant_decode_attention_gb300 import api
    api.nvfp4_logits(s["x"], prompt=s["prompt"], prompt_lens=s["prompt_lens"], output=s["output"],
                     output_lens=s["output_lens"], repetition=s["repetition"], frequency=s["frequency"],
                     presence=s["presence"], bias_tokens=s["bias_tokens"], bias_values=s["bias_values"],
                     bias_lens=s["bias_lens"], mask=s["mask"], mask_ids=s["mask_ids"], out=s["out"],
                     tokens=s["tokens"])
    return {"logits": s["out"], "tokens": s["tokens"]}


def _e2m1_bytes():
    """For each byte of two E2M1 codes, the two values as E4M3 bytes (both
    types hold the eight magnitudes), for reading an NVFP4 cache's values."""
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
    one = mags.to(torch.float8_e4m3fn).view(torch.uint8)
    two = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)
    return two.view(torch.int16).reshape(256).cuda()


def _nvfp4_parts(s, name):
    m = s["total"] * s["case"]["H_kv"] * s["case"]["D"]
    return s[name][:m // 2], s[name][m // 2:]


def _append_outputs(s):
    """The whole caches and the rotated queries; an NVFP4 cache as the values
    that its codes and its block scales stand for."""
    if s["case"]["kv"] != "nvfp4":
        return {"k": s["k"], "v": s["v"], "q": s["q_out"]}
    r = {"q": s["q_out"]}
    for name in ("k", "v"):
        codes, blocks = _nvfp4_parts(s, name)
        r[name + "_codes"] = s["e2m1_bytes"].index_select(0, codes.int()).view(torch.float8_e4m3fn)
        r[name + "_blocks"] = blocks.view(torch.float8_e4m3fn)
    return r


def _turn(x, cos, sin, c):
    """x [n, H, D] fp32 with dims [offset, offset + rope_dim) rotated."""
    o, d = c["rope_offset"], c["rope_dim"]
    part = x[..., o:o + d]
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = part[..., :d // 2], part[..., d // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([x[..., :o], turned, x[..., o + d:]], -1)


def _plain_append(s):
    c, live = s["case"], s["live"]
    angle = s["positions"][:live, None].double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    s["q_out"][:live] = _turn(s["q"][:live].float(), cos, sin, c).to(BF16)
    for name, new, scale in (("k", s["k_new"], s["k_scale"]), ("v", s["v_new"], s["v_scale"])):
        if new is None:
            continue
        x = new[:live].float()
        if name == "k":
            x = _turn(x, cos, sin, c)
        if c["kv"] == "bf16":
            s[name].view(-1, c["H_kv"], c["D"])[s["entry"]] = x.to(BF16)
        elif c["kv"] == "e4m3":
            stored = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[name].view(torch.uint8).view(-1, c["H_kv"], c["D"])[s["entry"]] = stored.view(torch.uint8)
        else:
            b = x.view(live, c["H_kv"], c["D"] // 16, 16)
            blocks = (b.abs().amax(-1) / (6 * scale)).clamp(max=448).to(torch.float8_e4m3fn)
            step = (blocks.float() * scale)[..., None]
            u = torch.where(step > 0, b / step, torch.zeros_like(b))
            a = u.abs()  # nearest of 0, .5, 1, 1.5, 2, 3, 4, 6; ties to the even code
            code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
            code = torch.where(torch.signbit(u), code + 8, code).view(live, c["H_kv"], c["D"])
            packed = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
            codes_all, blocks_all = _nvfp4_parts(s, name)
            codes_all.view(-1, c["H_kv"], c["D"] // 2)[s["entry"]] = packed
            blocks_all.view(-1, c["H_kv"], c["D"] // 16)[s["entry"]] = blocks.view(torch.uint8)
    return _append_outputs(s)


def _plain_adapters(s):
    """All rows through all adapters side by side; a row keeps its own part."""
    c = s["case"]
    count, rank, K, N = c["count"], c["rank"], c["K"], c["N"]
    x = s["x"].to(BF16).float()
    t = (x @ s["a"].float().view(count * rank, K).T).view(-1, count, rank)
    mine = s["ids"][:, None] == torch.arange(count, device="cuda", dtype=torch.int32)
    inside = torch.arange(rank, device="cuda") < s["ranks"][:, None]
    t = torch.where(mine[..., None] & inside, t * s["scales"][:, None], torch.zeros_like(t))
    y = s["y"] + t.view(-1, count * rank) @ s["b"].float().permute(0, 2, 1).reshape(count * rank, N)
    return {"y": y, "y_bf16": y.to(BF16) if c["y"] == "both" else None}


def _plain_logits(s):
    c = s["case"]
    B, V = c["B"], c["V"]

    def counts(tokens, lens):
        live = torch.arange(tokens.shape[1], device="cuda") < lens[:, None]
        at = torch.where(live, tokens, torch.full_like(tokens, V)).long()
        return torch.zeros((B, V + 1), device="cuda").scatter_add_(1, at, live.float())[:, :V]

    l = s["x"].float()
    made = counts(s["output"], s["output_lens"])
    seen = (made + counts(s["prompt"], s["prompt_lens"])) > 0
    rep = s["repetition"][:, None]
    l = torch.where(seen, torch.where(l > 0, l / rep, l * rep), l)
    l = l - s["frequency"][:, None] * made
    l = l - s["presence"][:, None] * (made > 0).float()
    if s["bias_tokens"] is not None:  # a row's bias tokens are distinct
        live = torch.arange(s["bias_tokens"].shape[1], device="cuda") < s["bias_lens"][:, None]
        at = torch.where(live, s["bias_tokens"], torch.full_like(s["bias_tokens"], V)).long()
        bias = torch.zeros((B, V + 1), device="cuda").scatter_(1, at, s["bias_values"])[:, :V]
        l = l + bias
    if s["mask"] is not None:
        v = torch.arange(V, device="cuda")
        word = s["mask"][s["mask_ids"].clamp(min=0)][:, v // 32]
        allowed = ((word >> (v % 32).int()) & 1) != 0
        allowed = allowed | (s["mask_ids"] < 0)[:, None]
        l = torch.where(allowed, l, torch.full_like(l, -math.inf))
    best = torch.where(l.isnan(), torch.full_like(l, -math.inf), l).amax(-1, keepdim=True)
    first = torch.where(l == best, torch.arange(V, device="cuda", dtype=torch.int32), V).amin(-1)
    token = torch.where(best[:, 0] > -math.inf, first, -1).to(torch.int32)
    return {"logits": l if c["write"] else None, "tokens": token}


# ------------------------------------------------------------------ work

def work(c):
    if c["op"] == "append":
        live, e = c["n"] - c["pad"], {"bf16": 2, "fp32": 4}[c["x"]]
        stored = {"bf16": 2.0, "e4m3": 1.0, "nvfp4": 9 / 16}[c["kv"]]
        kv_rows = c["H_kv"] * (1 if c["latent"] else 2)
        per = c["D"] * (c["H_q"] * (e + 2) + kv_rows * (e + stored)) + 8
        turned = (c["H_q"] + c["H_kv"]) * c["rope_dim"]
        return {"bytes": live * per, "flops": live * 3 * turned}
    if c["op"] == "adapters":
        ids, ranks = _adapter_of(c), np.array(_ranks(c))
        used = ranks[np.unique(ids[ids >= 0])].sum()
        rank_rows = ranks[ids[ids >= 0]].sum()
        per = c["K"] * {"bf16": 2, "fp32": 4}[c["x"]] + 8 * c["N"] + (2 * c["N"] if c["y"] == "both" else 0) + 4
        return {"bytes": int(c["n"] * per + 2 * used * (c["K"] + c["N"])),
                "flops": int(2 * rank_rows * (c["K"] + c["N"]))}
    B, V = c["B"], c["V"]
    per = V * {"bf16": 2, "fp32": 4}[c["x"]] + (4 * V if c["write"] else 0)
    lists = 4 * 0.6 * c["history"] + 8 * 0.6 * c["biases"]
    masks = min(B, 4) * V / 8 if c["mask"] else 0
    return {"bytes": int(B * (per + lists) + masks), "flops": 2 * B * V}


# ------------------------------------------------------------------ exact values

def exact(case, seed):
    """What run() returns, from each definition in 64 bits: bf16 and E4M3
    results before their rounding, NVFP4 scales and codes with it (they are
    what the definition says is stored)."""
    s = prepare(case, seed)
    return {"append": _exact_append, "adapters": _exact_adapters, "logits": _exact_logits}[case["op"]](s)


def _exact_append(s):
    c, live = s["case"], s["live"]
    o, d = c["rope_offset"], c["rope_dim"]
    phase = torch.polar(torch.ones((live, 1, d // 2), dtype=torch.float64, device="cuda"),
                        torch.outer(s["positions"][:live].double(), s["inv_freq"].double())[:, None])

    def turned(x):
        x = x[:live].double().clone()
        lo, hi = (x[..., o:o + d:2], x[..., o + 1:o + d:2]) if c["interleaved"] else (
            x[..., o:o + d // 2], x[..., o + d // 2:o + d])
        z = torch.complex(lo.contiguous(), hi.contiguous()) * phase
        lo.copy_(z.real)
        hi.copy_(z.imag)
        return x

    q = s["q_out"].double()
    q[:live] = turned(s["q"])
    r = {"q": q}
    for name, x, scale in (("k", turned(s["k_new"]), s["k_scale"]), ("v", s["v_new"], s["v_scale"])):
        if x is None:
            r[name] = None
            continue
        x = x[:live].double()
        if c["kv"] != "nvfp4":
            cache = s[name].double()
            if c["kv"] == "e4m3":
                x = torch.clip(x / scale, -448.0, 448.0)
            cache.view(-1, c["H_kv"], c["D"])[s["entry"]] = x
            r[name] = cache
            continue
        m = s["total"] * c["H_kv"] * c["D"]
        blocks = s[name][m // 2:].view(torch.float8_e4m3fn).double().view(-1, c["H_kv"], c["D"] // 16)
        codes = s["e2m1_bytes"][s[name][:m // 2].long()].view(torch.float8_e4m3fn).double()
        codes = codes.view(-1, c["H_kv"], c["D"])
        groups = x.unflatten(-1, (-1, 16))
        want = groups.abs().amax(-1) / (6 * scale)
        block = torch.minimum(want, torch.full_like(want, 448.0)).float().to(torch.float8_e4m3fn).double()
        grid = torch.tensor([0, 1, 2, 4, 6, 0.5, 1.5, 3], dtype=torch.float64, device="cuda")  # even codes first
        ratio = torch.nan_to_num(groups.abs() / (block * scale)[..., None])
        near = grid[(ratio[..., None] - grid).abs().argmin(-1)]
        blocks[s["entry"]] = block
        codes[s["entry"]] = (near * groups.sign()).flatten(-2)
        r[name + "_codes"], r[name + "_blocks"] = codes.reshape(-1), blocks.reshape(-1)
    return r


def _exact_adapters(s):
    y = s["y"].double()
    x = s["x"].to(BF16).double()
    ranks, ids = s["ranks"].tolist(), s["ids"].cpu().numpy()
    for a, r in enumerate(ranks):
        rows = torch.tensor(np.flatnonzero(ids == a), device="cuda")
        low = x[rows] @ s["a"][a, :r].double().T
        y[rows] += s["scales"][a].double() * (low @ s["b"][a, :, :r].double().T)
    return {"y": y, "y_bf16": y.clone() if s["case"]["y"] == "both" else None}


def _exact_logits(s):
    c = s["case"]
    lines, picks = [], []
    lens = {k: s[k].tolist() for k in ("prompt_lens", "output_lens")}
    blens = s["bias_lens"].tolist() if s["bias_lens"] is not None else None
    mids = s["mask_ids"].tolist() if s["mask_ids"] is not None else None
    for b in range(c["B"]):
        l = s["x"][b].double()
        made = torch.bincount(s["output"][b, :lens["output_lens"][b]], minlength=c["V"]).double()
        told = torch.bincount(s["prompt"][b, :lens["prompt_lens"][b]], minlength=c["V"])
        factor = torch.where(l > 0, 1 / s["repetition"][b].double(), s["repetition"][b].double())
        l = l * torch.where((made > 0) | (told > 0), factor, torch.ones_like(factor))
        l = l - made * s["frequency"][b].double() - made.clamp(max=1) * s["presence"][b].double()
        if blens is not None:
            m = blens[b]
            l.index_add_(0, s["bias_tokens"][b, :m].long(), s["bias_values"][b, :m].double())
        if mids is not None and mids[b] >= 0:
            bits = np.unpackbits(s["mask"][mids[b]].cpu().numpy().astype("<i4").view(np.uint8), bitorder="little")
            l[torch.tensor(bits[:c["V"]] == 0, device="cuda")] = -math.inf
        lines.append(l)
        picks.append(int(l.argmax()) if float(l.max()) > -math.inf else -1)
    return {"logits": torch.stack(lines) if c["write"] else None,
            "tokens": torch.tensor(picks, dtype=torch.int32)}
