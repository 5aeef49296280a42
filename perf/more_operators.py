"""Cases, plain forms and exact values of four operators of a decode step over
drafted tokens:

* norm: queries and keys normed head by head, rotated and written into the cache
  (append with norms), drafted tokens at entries of their own;
* tree: attention of a tree of drafted tokens over the cache, with a sliding
  window and first tokens that stay visible where a layer has them;
* verify: drafted tokens accepted or not by the target's probabilities, and the
  next token, from given random numbers;
* move: cache entries of all layers -- pages copied for a fork, the entries of
  the accepted tokens moved to their places.

``listed()`` names the cases that are timed, ``draw(rng)`` gives others of the
same ranges; ``prepare``/``run`` make the inputs and do one pass, in plain
torch operations or (``own``) through the package's entry points.
"""

import math

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TYPES = {"bf16": BF16, "fp32": F32}


# ------------------------------------------------------------------ cases

def listed():
    gqa = dict(H_q=32, H_kv=8, D=128)
    return [
        # 64 requests' trees of 8 drafted tokens into an E4M3 cache, each at its own entry
        dict(name="norm_tree", op="norm", B=64, T=8, context=2048, layout="paged", page=16, kv="e4m3", x="fp32",
             rope_dim=128, interleaved=False, tree=True, **gqa),
        # prompts: 8192 new tokens in four runs
        dict(name="norm_prompt", op="norm", B=4, T=2048, context=4096, layout="paged", page=64, kv="bf16",
             x="bf16", rope_dim=128, interleaved=False, tree=False, **gqa),
        # one request, a small tree: nothing but latency
        dict(name="tree_1", op="tree", B=1, T=8, context=4096, pad=0, layout="paged", page=16, kv="bf16",
             window=0, sinks=0, tree=True, **gqa),
        # a step of 32 requests with up to 16 drafted tokens each
        dict(name="tree_32", op="tree", B=32, T=16, context=8192, pad=0, layout="paged", page=64, kv="bf16",
             window=0, sinks=0, tree=True, **gqa),
        # odd sizes, a 4-bit cache, padded rows
        dict(name="tree_7_nvfp4", op="tree", B=7, T=13, context=2999, pad=1, layout="paged", page=48, kv="nvfp4",
             window=0, sinks=0, tree=True, H_q=20, H_kv=4, D=64),
        # wide trees of 64 tokens: the tensor cores' work counts
        dict(name="tree_wide", op="tree", B=8, T=64, context=16384, pad=0, layout="contiguous", page=0, kv="bf16",
             window=0, sinks=0, tree=True, H_q=64, H_kv=8, D=128),
        # a windowed layer's plain decode step over long E4M3 contexts
        dict(name="window_64", op="tree", B=64, T=1, context=32768, pad=0, layout="paged", page=16, kv="e4m3",
             window=4096, sinks=4, tree=False, **gqa),
        # one request's chain of three drafted tokens against its draft model's probabilities
        dict(name="verify_1", op="verify", B=1, T=4, V=32000, x="fp32", draft=True),
        # trees without draft probabilities, an odd vocabulary, bf16 logits
        dict(name="verify_32_tree", op="verify", B=32, T=16, V=50001, x="bf16", draft=False),
        # a large step: chains of seven drafted tokens
        dict(name="verify_64", op="verify", B=64, T=8, V=131072, x="fp32", draft=True),
        # accepted entries of 64 requests moved up in the caches of 32 layers
        dict(name="move_accepted", op="move", what="compact", B=64, T=16, context=128, layers=32, layout="paged",
             page=16, kv="bf16", **gqa),
        # 256 pages copied in the caches of 16 layers
        dict(name="move_pages", op="move", what="pages", B=256, T=0, context=0, layers=16, layout="paged", page=16,
             kv="bf16", **gqa),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _layout(rng):
    layout = rng.choice(["paged", "paged", "paged", "contiguous", "indexed"])
    return dict(layout=layout, page=rng.choice([1, 16, 48, 64, 128]) if layout == "paged" else 0)


def draw(rng):
    op = rng.choice(["norm", "tree", "tree", "verify", "move"])
    H_q, H_kv, D = rng.choice([(32, 8, 128), (8, 1, 64), (64, 8, 128), (20, 4, 64), (7, 7, 128), (48, 2, 128),
                               (32, 32, 128), (128, 8, 128)])
    heads = dict(H_q=H_q, H_kv=H_kv, D=D)
    if op == "norm":
        tree = rng.random() < 0.6
        most = 8192 * 48 * 128 // ((H_q + 2 * H_kv) * D)
        T = _log(rng, 1, 64) if tree else _log(rng, 64, min(2048, most))
        B = max(1, min(_log(rng, 1, 256) if tree else rng.randint(1, 4), most // T))
        return dict(op=op, B=B, T=T, context=max(2 * T, _log(rng, 64, 2048)), kv=rng.choice(["bf16", "e4m3", "nvfp4"]),
                    x=rng.choice(["bf16", "fp32"]), rope_dim=rng.choice([D, D, D // 2, 32]),
                    interleaved=rng.random() < 0.3, tree=tree, **_layout(rng), **heads)
    if op == "tree":
        T = _log(rng, 1, 64)
        window = rng.choice([0, 0, _log(rng, 1, 8192)])
        context = _log(rng, 1, 32768)
        seen = min(context, window + 64) if window else context
        B = _log(rng, 1, 256)
        while B > 1 and (B * context * H_kv * D > 64 * 32768 * 8 * 128 or B * seen * H_kv * D > 32 * 8192 * 8 * 128
                         or B * T * H_q * seen * D > 8 * 64 * 64 * 16384 * 128):
            B //= 2
        return dict(op=op, B=B, T=T, context=context, pad=rng.choice([0, 0, rng.randint(0, B // 4)]),
                    kv=rng.choice(["bf16", "bf16", "e4m3", "nvfp4"]), window=window,
                    sinks=rng.choice([0, 1, 4, 100]) if window else 0, tree=rng.random() < 0.7, **_layout(rng),
                    **heads)
    if op == "verify":
        V = _log(rng, 1000, 131072)
        T = _log(rng, 1, 32)
        B = min(_log(rng, 1, 256), max(1, 64 * 8 * 131072 // (T * V)))
        return dict(op=op, B=B, T=T, V=V, x=rng.choice(["bf16", "fp32"]), draft=rng.random() < 0.5)
    what = rng.choice(["compact", "pages"])
    layers = _log(rng, 1, 48)
    kv = rng.choice(["bf16", "e4m3"])
    if what == "compact":
        return dict(op=op, what=what, B=min(_log(rng, 1, 128), max(1, 64 * 32 * 8 * 128 // (layers * H_kv * D))),
                    T=rng.randint(2, 64), context=rng.randint(1, 128), layers=layers, kv=kv, **_layout(rng), **heads)
    page = rng.choice([16, 32, 48, 64])
    most = 256 * 16 * 16 * 8 * 128 // (layers * page * H_kv * D)
    return dict(op=op, what=what, B=max(1, min(_log(rng, 1, 256), most)), T=0, context=0, layers=layers,
                layout="paged", page=page, kv=kv, **heads)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, g, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32).to(dtype)


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return {"norm": _prepare_norm, "tree": _prepare_tree, "verify": _prepare_verify,
            "move": _prepare_move}[case["op"]](case, seed)


def _parents(rs, B, T, tree):
    """Each node's parent: an earlier node, more often a late one; a chain."""
    if not tree:
        return np.tile(np.arange(-1, T - 1), (B, 1))
    at = np.floor(rs.random_sample((B, T)) ** 0.5 * np.arange(T)).astype(np.int64)
    return np.where(np.arange(T) == 0, -1, np.minimum(at, np.arange(T) - 1))


def _depths(parents):
    d = np.zeros_like(parents)
    for t in range(1, parents.shape[1]):
        d[:, t] = np.take_along_axis(d, parents[:, t:t + 1], 1)[:, 0] + 1
    return d


def _places(c, rs, need):
    """A cache's leading sizes, the rows' table and the entry that row b's
    list has at place j: rows of `need` places at most, pages in any order."""
    B, page = c["B"], max(c["page"], 1)
    if c["layout"] == "contiguous":
        return (B, need), None, np.arange(B)[:, None] * need + np.arange(need)
    width = -(-need // page)
    pages = B * width + 3
    table = rs.permutation(pages)[:B * width].reshape(B, width)
    lead = (pages, page) if c["layout"] == "paged" else (pages,)
    j = np.arange(need)
    return lead, table, table[:, j // page] * page + j % page


def _cache(c, g, entries, lead):
    """K or V with what it already holds, values of size 1 once scaled."""
    H, D = c["H_kv"], c["D"]
    if c["kv"] == "bf16":
        return _randn((*lead, H, D), g, BF16)
    if c["kv"] == "e4m3":
        return (_randn((*lead, H, D), g) * 16).to(torch.float8_e4m3fn)
    m = entries * H * D  # codes of all entries, then their block scales, in one buffer
    kv = torch.empty(m // 2 + m // 16, dtype=torch.uint8, device="cuda")
    kv[:m // 2] = torch.randint(0, 256, (m // 2,), generator=g, device="cuda", dtype=torch.uint8)
    kv[m // 2:] = torch.randint(32, 64, (m // 16,), generator=g, device="cuda", dtype=torch.uint8)
    return kv


def _problem(c, lead, width, scales):
    from invariant_decode_attention_gb300 import api
    return api.problem(batch=c["B"], num_q_heads=c["H_q"], num_kv_heads=c["H_kv"], head_dim_qk=c["D"],
                       layout=c["layout"], scale=c["D"] ** -0.5, page_size=c["page"], width=max(width, 1),
                       num_blocks=lead[0] if c["layout"] != "contiguous" else 0, k_scale=scales[0],
                       v_scale=scales[1], kv_dtype={"bf16": api.KV_BF16, "e4m3": api.KV_FP8_E4M3,
                                                    "nvfp4": api.KV_NVFP4}[c["kv"]])


def _prepare_norm(c, seed):
    """The fused projections of B runs of T new tokens after what their rows
    hold; a tree's token is rotated by its depth and stored by its number."""
    g, rs = _gen(seed), np.random.RandomState(seed % (1 << 31))
    B, T, H_q, H_kv, D = c["B"], c["T"], c["H_q"], c["H_kv"], c["D"]
    n, x_type = B * T, TYPES[c["x"]]
    qkv = _randn((n, (H_q + 2 * H_kv) * D), g, x_type)
    need = c["context"] + T
    lead, table, entry = _places(c, rs, need)
    start = rs.randint(0, c["context"] + 1, B)
    at = start[:, None] + np.arange(T)
    positions = start[:, None] + _depths(_parents(rs, B, T, c["tree"]))
    rows = np.repeat(np.arange(B), T)
    entry = np.take_along_axis(entry, at, 1).reshape(-1)
    total = int(np.prod(lead))
    half = c["rope_dim"] // 2
    inv_freq = (10000.0 ** (-torch.arange(half, dtype=F64) / half)).float().cuda()
    scales = (1.0 / 64, 1.0 / 48)
    s = dict(case=c, q=qkv[:, :H_q * D].view(n, H_q, D), k_new=qkv[:, H_q * D:(H_q + H_kv) * D].view(n, H_kv, D),
             v_new=qkv[:, (H_q + H_kv) * D:].view(n, H_kv, D), k=_cache(c, g, total, lead),
             v=_cache(c, g, total, lead), q_weight=_randn((D,), g, BF16) * 0.1 + 1, k_weight=_randn((D,), g, BF16) * 0.1 + 1,
             eps=1e-6, inv_freq=inv_freq, positions=_i32(positions.reshape(-1)), total=total, scales=scales,
             entry=torch.tensor(entry, device="cuda"), table=None if table is None else _i32(table),
             rows=_i32(entry if c["layout"] == "indexed" else rows),
             entries=_i32(at.reshape(-1)) if c["layout"] != "indexed" else None,
             q_out=torch.zeros((n, H_q, D), dtype=BF16, device="cuda"),
             e2m1_bytes=_e2m1_bytes() if c["kv"] == "nvfp4" else None)
    if own:  # what a server makes once: the problem's description, the rotation's and the norms'
        from invariant_decode_attention_gb300 import api
        s["prob"] = _problem(c, lead, need if table is None else table.shape[1], scales)
        s["rope"] = api.rope(inv_freq, interleaved=c["interleaved"])
        s["norm"] = api.head_norm(s["q_weight"], s["k_weight"], eps=s["eps"])
    return s


def _prepare_tree(c, seed):
    """Contexts of ragged lengths, then the drafted tokens' own entries; the
    last `pad` rows are padding and have none."""
    g, rs = _gen(seed), np.random.RandomState(seed % (1 << 31))
    B, T, H_q, D, live = c["B"], c["T"], c["H_q"], c["D"], c["B"] - c["pad"]
    need = c["context"] + T
    lead, table, entry = _places(c, rs, need)
    total = int(np.prod(lead))
    counts = rs.randint(max(1, T // 2), T + 1, B)
    lengths = rs.randint(c["context"] // 2, c["context"] + 1, B)
    counts[live:] = lengths[live:] = 0
    scales = (1.0, 1.0) if c["kv"] == "bf16" else (1.0 / 16, 1.0 / 16) if c["kv"] == "e4m3" else (0.5, 0.5)
    parents = _parents(rs, B, T, c["tree"])
    s = dict(case=c, q=_randn((B, T, H_q, D), g, BF16) * 2, k=_cache(c, g, total, lead), v=_cache(c, g, total, lead),
             lengths=_i32(lengths), counts=_i32(counts), parents=_i32(parents) if c["tree"] else None, table=None,
             par=torch.tensor(parents, device="cuda"), depth=torch.tensor(_depths(parents), device="cuda"),
             entry=torch.tensor(entry, device="cuda"), total=total, scales=scales,
             out=torch.zeros((B, T, H_q, D), dtype=BF16, device="cuda"), lse=torch.zeros((B, T, H_q), device="cuda"))
    if table is not None:
        s["table"] = _i32(table)
    if own:  # what a server makes once: the problem's description and the workspace
        from invariant_decode_attention_gb300 import api
        s["prob"] = _problem(c, lead, need if table is None else table.shape[1], scales)
        s["ws"] = api.tree_workspace(s["prob"], T)
    return s


def _prepare_verify(c, seed):
    """The target's logits at every node and tokens drafted by a model near it:
    drawn from its probabilities (chains), or likely ones (trees).  Every eighth
    row decodes greedily."""
    g, rs = _gen(seed), np.random.RandomState(seed % (1 << 31))
    B, T, V = c["B"], c["T"], c["V"]
    logits = (_randn((B, T, V), g) * 3).to(TYPES[c["x"]])
    parents = _parents(rs, B, T, not c["draft"])
    par = torch.tensor(parents, device="cuda").clamp(min=0)
    near = torch.gather(logits.float(), 1, par[:, :, None].expand(B, T, V)) + _randn((B, T, V), g) * 0.5
    draft = torch.softmax(near, -1)
    race = torch.empty_like(draft).exponential_(generator=g)
    tokens = (draft / race).argmax(-1).to(torch.int32)
    tau = np.where(np.arange(B) % 8 == 7, 0.0, rs.choice([0.7, 1.0, 1.3], B))
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(case=c, logits=logits, tokens=tokens, parents=None if c["draft"] else _i32(parents),
             par=torch.tensor(parents, device="cuda"), draft=draft if c["draft"] else None,
             counts=_i32(rs.randint(max(1, T // 2), T + 1, B)),
             temperature=torch.tensor(tau, dtype=F32, device="cuda"),
             uniforms=torch.rand((B, T), generator=g, device="cuda"), final=torch.rand(B, generator=g, device="cuda"),
             accepted=torch.zeros(B, **i32), nodes=torch.zeros((B, T), **i32), out=torch.zeros((B, T), **i32))
    if own:  # what a server makes once: the workspace
        from invariant_decode_attention_gb300 import api
        s["ws"] = api.verify_workspace(B, T, V)
    return s


def _prepare_move(c, seed):
    """The caches of all layers, and which of a row's nodes were accepted (each
    where it belongs already, or from behind all places that are filled) or which
    pages go where."""
    g, rs = _gen(seed), np.random.RandomState(seed % (1 << 31))
    B, T, layers, H, D = c["B"], c["T"], c["layers"], c["H_kv"], c["D"]
    s = dict(case=c, table=None)
    if c["what"] == "pages":
        lead = (4 * B, c["page"])
        order = rs.permutation(4 * B)
        width = 1
        s.update(src=_i32(order[rs.randint(0, B, B)]), dst=_i32(order[B:2 * B]))
    else:
        lead, table, entry = _places(c, rs, c["context"] + T)
        width = c["context"] + T if table is None else table.shape[1]
        lengths = rs.randint(0, c["context"] + 1, B)
        accepted = rs.randint(0, max(1, T // 2), B)
        nodes = np.full((B, T), -1)
        src, dst = [], []
        for b in range(B):
            m = accepted[b] + 1
            same = rs.randint(1, m + 1)  # the first so many stay where they are
            late = np.sort(rs.choice(np.arange(m, T), m - same, replace=False))
            nodes[b, :m] = np.concatenate([np.arange(same), late])
            src.append(entry[b, lengths[b] + nodes[b, :m]])
            dst.append(entry[b, lengths[b] + np.arange(m)])
        s.update(lengths=_i32(lengths), nodes=_i32(nodes), accepted=_i32(accepted),
                 table=None if table is None else _i32(table), new_lengths=torch.zeros_like(_i32(lengths)),
                 src=torch.tensor(np.concatenate(src), device="cuda"),
                 dst=torch.tensor(np.concatenate(dst), device="cuda"))
    for name in ("k", "v"):
        x = torch.empty((layers, *lead, H, D), dtype=BF16 if c["kv"] == "bf16" else torch.float8_e4m3fn, device="cuda")
        for layer in range(layers):
            x[layer] = _randn((*lead, H, D), g).to(x.dtype)
        s[name] = x
    if own:  # what a server makes once: the problem's description and the layers' caches
        from invariant_decode_attention_gb300 import api
        s["prob"] = _problem(c, lead, width, (1.0, 1.0))
        s["caches"] = api.Caches(s["prob"], list(s["k"]), list(s["v"]))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm": _own_norm, "tree": _own_tree, "verify": _own_verify, "move": _own_move}[op](s)
    return {"norm": _plain_norm, "tree": _plain_tree, "verify": _plain_verify, "move": _plain_move}[op](s)


def _own_norm(s):
    from invariant_decode_attention_gb300 import api
    api.append(s["prob"], s["rope"], s["k_new"], s["v_new"], s["k"], s["v"], s["positions"], rows=s["rows"],
               table=s["table"] if s["case"]["layout"] == "paged" else None, q_new=s["q"], q_out=s["q_out"],
               norm=s["norm"], entries=s["entries"])
    return _norm_outputs(s)


def _own_tree(s):
    from invariant_decode_attention_gb300 import api
    c = s["case"]
    api.tree(s["prob"], s["q"], s["k"], s["v"], s["lengths"], parents=s["parents"], counts=s["counts"],
             table=s["table"], window=c["window"], sinks=c["sinks"], out=s["out"], lse=s["lse"], ws=s["ws"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_verify(s):
    from invariant_decode_attention_gb300 import api
    api.nvfp4_verify(s["logits"], s["tokens"], s["uniforms"], s["final"], parents=s["parents"], counts=s["counts"],
                     draft=s["draft"], temperature=s["temperature"], accepted=s["accepted"], nodes=s["nodes"],
                     out=s["out"], ws=s["ws"])
    return {"accepted": s["accepted"], "nodes": s["nodes"], "tokens": s["out"]}


def _own_move(s):
    from invariant_decode_attention_gb300 import api
    if s["case"]["what"] == "pages":
        api.copy_pages(s["prob"], s["caches"], s["src"], s["dst"])
        return {"k": s["k"], "v": s["v"]}
    api.compact(s["prob"], s["caches"], s["lengths"], s["nodes"], s["accepted"], table=s["table"],
                new_lengths=s["new_lengths"])
    return {"k": s["k"], "v": s["v"], "lengths": s["new_lengths"]}


def _e2m1_bytes():
    """For each byte of two E2M1 codes, the two values as E4M3 bytes (both
    types hold the eight magnitudes)."""
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
    one = mags.to(torch.float8_e4m3fn).view(torch.uint8)
    two = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)
    return two.view(torch.int16).reshape(256).cuda()


def _nvfp4_parts(s, name):
    m = s["total"] * s["case"]["H_kv"] * s["case"]["D"]
    return s[name][:m // 2], s[name][m // 2:]


def _norm_outputs(s):
    """The whole caches and the queries; an NVFP4 cache as the values that its
    codes and its block scales stand for."""
    if s["case"]["kv"] != "nvfp4":
        return {"k": s["k"], "v": s["v"], "q": s["q_out"]}
    r = {"q": s["q_out"]}
    for name in ("k", "v"):
        codes, blocks = _nvfp4_parts(s, name)
        r[name + "_codes"] = s["e2m1_bytes"].index_select(0, codes.int()).view(torch.float8_e4m3fn)
        r[name + "_blocks"] = blocks.view(torch.float8_e4m3fn)
    return r


def _plain_norm(s):
    c, n = s["case"], s["q"].shape[0]
    d = c["rope_dim"]
    angle = s["positions"][:, None].double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def normed(x, weight):
        x = x.float()
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()

    def turned(x):
        part = x[..., :d]
        if c["interleaved"]:
            a, b = part[..., 0::2], part[..., 1::2]
            part = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = part[..., :d // 2], part[..., d // 2:]
            part = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([part, x[..., d:]], -1)

    s["q_out"].copy_(turned(normed(s["q"], s["q_weight"])))
    for name, x, scale in (("k", turned(normed(s["k_new"], s["k_weight"])), s["scales"][0]),
                           ("v", s["v_new"].float(), s["scales"][1])):
        if c["kv"] == "bf16":
            s[name].view(-1, c["H_kv"], c["D"])[s["entry"]] = x.to(BF16)
        elif c["kv"] == "e4m3":
            stored = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[name].view(torch.uint8).view(-1, c["H_kv"], c["D"])[s["entry"]] = stored.view(torch.uint8)
        else:
            b = x.reshape(n, c["H_kv"], c["D"] // 16, 16)
            blocks = (b.abs().amax(-1) / (6 * scale)).clamp(max=448).to(torch.float8_e4m3fn)
            step = (blocks.float() * scale)[..., None]
            u = torch.where(step > 0, b / step, torch.zeros_like(b))
            a = u.abs()  # nearest of 0, .5, 1, 1.5, 2, 3, 4, 6; ties to the even code
            code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5))
            code = torch.where(torch.signbit(u), code + 8, code).view(n, c["H_kv"], c["D"])
            packed = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
            codes_all, blocks_all = _nvfp4_parts(s, name)
            codes_all.view(-1, c["H_kv"], c["D"] // 2)[s["entry"]] = packed
            blocks_all.view(-1, c["H_kv"], c["D"] // 16)[s["entry"]] = blocks.view(torch.uint8)
    return _norm_outputs(s)


def _values(s, name, scale, entry, dtype):
    """Cache entries [..., H_kv, D] of the given type."""
    c = s["case"]
    H, D = c["H_kv"], c["D"]
    if c["kv"] == "bf16":
        return s[name].view(-1, H, D)[entry].to(dtype)
    if c["kv"] == "e4m3":
        return s[name].view(torch.uint8).view(-1, H, D)[entry].view(torch.float8_e4m3fn).to(dtype) * scale
    codes, blocks = _nvfp4_parts(s, name)
    codes = codes.view(-1, H, D // 2)[entry]
    blocks = blocks.view(-1, H, D // 16)[entry].view(torch.float8_e4m3fn).to(dtype)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device="cuda")
    x = grid[torch.stack([codes & 15, codes >> 4], -1).int()].flatten(-2)
    return x * blocks.repeat_interleave(16, -1) * scale


def _plain_tree(s):
    """All rows padded to the longest; scores of what a node does not see -inf.
    With a window only the places that some node may see are gathered."""
    c = s["case"]
    B, T, H_q, H, D, W = c["B"], c["T"], c["H_q"], c["H_kv"], c["D"], c["window"]
    need = c["context"] + T
    L = s["lengths"].long()[:, None]
    j = torch.arange(need, device="cuda").expand(B, need)
    if W and W + T + c["sinks"] < need:
        first = torch.arange(c["sinks"], device="cuda").expand(B, -1)
        start = torch.clamp(L - W + 1, min=c["sinks"])
        last = start + torch.arange(W + T - 1, device="cuda")
        j = torch.cat([first, last], 1)
    there = j < L + s["counts"].long()[:, None]
    j = j.clamp(max=need - 1)
    entry = torch.gather(s["entry"], 1, j)
    k = _values(s, "k", s["scales"][0], entry, F32)  # [B, J, H, D]
    v = _values(s, "v", s["scales"][1], entry, F32)
    node = j - L  # the node at a place, negative: context
    pos = L + s["depth"]  # [B, T]
    step = torch.eye(T, device="cuda") + (s["par"][..., None] == torch.arange(T, device="cuda")).float()
    for _ in range(max(T - 1, 0).bit_length()):  # a node sees its parent, that one's parent, ...
        step = (step @ step).clamp(max=1)
    anc = step > 0
    at = node.clamp(0, T - 1)
    sees = torch.where((node >= 0)[:, None], torch.gather(anc, 2, at[:, None].expand(B, T, -1)), there[:, None])
    j_pos = torch.where(node >= 0, torch.gather(pos, 1, at), j)[:, None]
    sees = sees & there[:, None]
    if W:
        sees = sees & ((pos[..., None] - j_pos < W) | (j_pos < c["sinks"]))
    q = s["q"].float().view(B, T, H, H_q // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * (H_q // H), D)
    score = (q @ k.permute(0, 2, 3, 1)).view(B, H, T, H_q // H, -1) * D ** -0.5
    score = score.masked_fill(~sees[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top.isinf(), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, H, T * (H_q // H), -1) @ v.permute(0, 2, 1, 3)).view(B, H, T, H_q // H, D) / total
    lse = (top + total.log()).squeeze(-1)
    o, lse = o.permute(0, 2, 1, 3, 4).reshape(B, T, H_q, D), lse.permute(0, 2, 1, 3).reshape(B, T, H_q)
    mine = (torch.arange(T, device="cuda") < s["counts"][:, None])[..., None]
    s["out"].copy_(torch.where(mine[..., None], o.to(BF16), s["out"]))
    s["lse"].copy_(torch.where(mine, lse, s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _plain_verify(s):
    """In 64 bits: a token next to a border is one or the other."""
    c = s["case"]
    B, T, V = c["B"], c["T"], c["V"]
    x = s["logits"].double()
    tau = s["temperature"].double()[:, None]
    greedy = tau[:, 0] == 0
    top = x.amax(-1, keepdim=True)
    first = torch.where(x == top, torch.arange(V, device="cuda"), V).amin(-1)  # [B, T]
    warm = torch.where(tau > 0, tau, torch.ones_like(tau))[..., None]
    p = torch.exp((x - top) / warm)
    p = p / p.sum(-1, keepdim=True)
    t = torch.arange(T, device="cuda")
    tokens, par = s["tokens"].long(), s["par"]
    live = t < s["counts"][:, None]
    mine = torch.gather(p.flatten(1), 1, par.clamp(min=0) * V + tokens)  # a node's token by its parent's row
    right = torch.gather(first, 1, par.clamp(min=0)) == tokens
    again = (tokens[:, :, None] == tokens[:, None]) & (par[:, :, None] == par[:, None]) & (t[:, None] > t) & live[:, None]
    u, cur = s["uniforms"].double(), torch.zeros(B, dtype=torch.long, device="cuda")
    went = torch.ones(B, dtype=torch.bool, device="cuda")
    accepted = torch.zeros(B, dtype=torch.int32, device="cuda")
    nodes = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    nodes[:, 0] = 0
    for step in range(1, T):
        child = (par == cur[:, None]) & live & (t > 0)
        here = torch.gather(u, 1, cur[:, None])
        if c["draft"]:
            q = torch.gather(s["draft"].flatten(1), 1, t * V + tokens).double()
            take = here * q < mine
        else:
            take = here < torch.cumsum(torch.where(child & ~again.any(-1), mine, 0.0), 1)
        take = child & torch.where(greedy[:, None], right, take)
        went = went & take.any(1)
        cur = torch.where(went, torch.where(take, t, T).amin(1), cur)
        accepted += went.int()
        nodes[:, step] = torch.where(went, cur, -1).to(torch.int32)
    rest = torch.gather(p, 1, cur[:, None, None].expand(B, 1, V))[:, 0]
    child = (par == cur[:, None]) & live & (t > 0)
    if c["draft"]:  # a chain's next token was refused, or there is none
        q = torch.gather(s["draft"], 1, (cur + 1).clamp(max=T - 1)[:, None, None].expand(B, 1, V))[:, 0].double()
        less = (rest - q).clamp(min=0)
        rest = torch.where(child.any(1, keepdim=True) & (less.sum(1, keepdim=True) > 0), less, rest)
    else:
        gone = torch.zeros((B, V + 1), dtype=torch.bool, device="cuda")
        gone.scatter_(1, torch.where(child, tokens, V), True)
        rest = rest.masked_fill(gone[:, :V], 0.0)
    total = torch.cumsum(rest, 1)
    pick = (total > s["final"].double()[:, None] * total[:, -1:]).int().argmax(1)
    pick = torch.where(greedy, torch.gather(first, 1, cur[:, None])[:, 0], pick).to(torch.int32)
    out = torch.where(nodes[:, 1:] >= 0, torch.gather(s["tokens"], 1, nodes[:, 1:].clamp(min=0).long()), -1)
    out = torch.cat([out, torch.full((B, 1), -1, dtype=torch.int32, device="cuda")], 1)
    out.scatter_(1, accepted[:, None].long(), pick[:, None])
    return {"accepted": accepted, "nodes": nodes, "tokens": out}


def _plain_move(s):
    c = s["case"]
    for name in ("k", "v"):
        x = s[name].view(torch.uint8)
        if c["what"] == "pages":
            x[:, s["dst"].long()] = x[:, s["src"].long()]
        else:
            x = x.view(c["layers"], -1, x.shape[-2] * x.shape[-1])
            x[:, s["dst"]] = x[:, s["src"]]
    if c["what"] == "pages":
        return {"k": s["k"], "v": s["v"]}
    s["new_lengths"].copy_(s["lengths"] + s["accepted"] + 1)
    return {"k": s["k"], "v": s["v"], "lengths": s["new_lengths"]}


# ------------------------------------------------------------------ work

def work(c):
    stored = {"bf16": 2.0, "e4m3": 1.0, "nvfp4": 9 / 16}[c["kv"]] if "kv" in c else 0
    if c["op"] == "norm":
        n, e = c["B"] * c["T"], {"bf16": 2, "fp32": 4}[c["x"]]
        per = c["D"] * (c["H_q"] * (e + 2) + 2 * c["H_kv"] * (e + stored)) + 12
        return {"bytes": n * per, "flops": n * (c["H_q"] + c["H_kv"]) * (4 * c["D"] + 3 * c["rope_dim"])}
    if c["op"] == "tree":  # lengths and counts are 0.75 of the largest in the mean
        T, live = c["T"], c["B"] - c["pad"]
        nodes = (max(1, T // 2) + T) / 2
        context = 0.75 * c["context"]
        seen = min(context, c["window"] + c["sinks"]) if c["window"] else context
        kv = live * (seen + nodes) * 2 * c["H_kv"] * c["D"] * stored
        rows = live * nodes * c["H_q"]
        return {"bytes": int(kv + rows * (4 * c["D"] + 4)), "flops": int(4 * rows * c["D"] * (seen + nodes / 2))}
    if c["op"] == "verify":
        nodes = (max(1, c["T"] // 2) + c["T"]) / 2
        rows = c["B"] * nodes * c["V"]
        q = 4 * c["B"] * c["V"] if c["draft"] else 0
        return {"bytes": int(rows * {"bf16": 2, "fp32": 4}[c["x"]] + q), "flops": int(3 * rows)}
    entry = 2 * c["H_kv"] * c["D"] * stored * c["layers"]
    if c["what"] == "pages":
        return {"bytes": int(2 * c["B"] * c["page"] * entry), "flops": 0}
    moved = c["B"] * max(1.0, (c["T"] // 2) / 4)  # about half of the accepted are there already
    return {"bytes": int(2 * moved * entry), "flops": 0}


# ------------------------------------------------------------------ exact values

def exact(case, seed):
    """What run() returns, from each definition in 64 bits: bf16 and E4M3
    results before their rounding, NVFP4 scales and codes with it (they are
    what the definition says is stored)."""
    s = prepare(case, seed)
    return {"norm": _exact_norm, "tree": _exact_tree, "verify": _exact_verify, "move": _exact_move}[case["op"]](s)


def _exact_norm(s):
    c, d = s["case"], s["case"]["rope_dim"]
    n = s["q"].shape[0]
    phase = torch.polar(torch.ones((n, 1, d // 2), dtype=F64, device="cuda"),
                        torch.outer(s["positions"].double(), s["inv_freq"].double())[:, None])

    def turned(x, weight):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + s["eps"]).sqrt() * weight.double()
        lo, hi = (x[..., 0:d:2], x[..., 1:d:2]) if c["interleaved"] else (x[..., :d // 2], x[..., d // 2:d])
        z = torch.complex(lo.contiguous(), hi.contiguous()) * phase
        lo.copy_(z.real)
        hi.copy_(z.imag)
        return x

    r = {"q": turned(s["q"], s["q_weight"])}
    for name, x, scale in (("k", turned(s["k_new"], s["k_weight"]), s["scales"][0]),
                           ("v", s["v_new"].double(), s["scales"][1])):
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
        grid = torch.tensor([0, 1, 2, 4, 6, 0.5, 1.5, 3], dtype=F64, device="cuda")  # even codes first
        ratio = torch.nan_to_num(groups.abs() / (block * scale)[..., None])
        near = grid[(ratio[..., None] - grid).abs().argmin(-1)]
        blocks[s["entry"]] = block
        codes[s["entry"]] = (near * groups.sign()).flatten(-2)
        r[name + "_codes"], r[name + "_blocks"] = codes.reshape(-1), blocks.reshape(-1)
    return r


def _exact_tree(s):
    """Row by row, each over the places that it has."""
    c = s["case"]
    T, H_q, H, D, W = c["T"], c["H_q"], c["H_kv"], c["D"], c["window"]
    out, lse = torch.zeros(s["out"].shape, dtype=F64, device="cuda"), torch.zeros(s["lse"].shape, dtype=F64, device="cuda")
    par, depth = s["par"].tolist(), s["depth"].tolist()
    for b, (L, n) in enumerate(zip(s["lengths"].tolist(), s["counts"].tolist())):
        if n == 0:
            continue
        low = max(0, L - W + 1) if W else 0
        places = np.concatenate([np.arange(min(low, c["sinks"])), np.arange(low, L + n)])
        sees = np.zeros((n, len(places)), dtype=bool)
        for t in range(n):
            pos = L + depth[b][t]
            place = np.where(places < L, places, -1)
            mine = place >= 0
            a = t
            while a >= 0:
                mine |= places == L + a
                place = np.where(places == L + a, L + depth[b][a], place)
                a = par[b][a]
            sees[t] = mine & ((place > pos - W) | (place < c["sinks"])) if W else mine
        entry = s["entry"][b][torch.tensor(places, device="cuda")]
        k = _values(s, "k", s["scales"][0], entry, F64)
        v = _values(s, "v", s["scales"][1], entry, F64)
        hide = ~torch.tensor(sees, device="cuda")
        for h in range(H):
            heads = slice(h * (H_q // H), (h + 1) * (H_q // H))
            score = torch.einsum("tgd,jd->gtj", s["q"][b, :n, heads].double(), k[:, h]) / math.sqrt(D)
            score = score.masked_fill(hide, -math.inf)
            z = torch.logsumexp(score, -1)
            lse[b, :n, heads] = z.T
            out[b, :n, heads] = torch.einsum("gtj,jd->tgd", torch.exp(score - z[..., None]), v[:, h])
    return {"out": out, "lse": lse}


def _exact_verify(s):
    c = s["case"]
    B, T, V = c["B"], c["T"], c["V"]
    par, tokens, counts = s["par"].tolist(), s["tokens"].tolist(), s["counts"].tolist()
    u, final, tau = s["uniforms"].tolist(), s["final"].tolist(), s["temperature"].tolist()
    accepted, nodes, out = np.zeros(B), np.full((B, T), -1), np.full((B, T), -1)

    def probabilities(b, t):
        x = s["logits"][b, t].double()
        return torch.softmax(x / tau[b], 0) if tau[b] else (torch.arange(V, device="cuda") == x.argmax()).double()

    for b in range(B):
        path = [0]
        while True:
            p = probabilities(b, path[-1])
            kids = [t for t in range(1, counts[b]) if par[b][t] == path[-1]]
            at, took = 0.0, None
            for i, t in enumerate(kids):
                token = tokens[b][t]
                if c["draft"] and tau[b]:
                    yes = u[b][path[-1]] * float(s["draft"][b, t, token]) < float(p[token])
                else:
                    at += float(p[token]) if token not in [tokens[b][k] for k in kids[:i]] else 0.0
                    yes = u[b][path[-1]] < at
                if yes:
                    took = t
                    break
            if took is None:
                break
            path.append(took)
        if kids and tau[b] and c["draft"]:
            less = torch.clamp(p - s["draft"][b, kids[0]].double(), min=0)
            p = less if float(less.sum()) > 0 else p
        elif kids and tau[b]:
            p[[tokens[b][t] for t in kids]] = 0
        total = torch.cumsum(p, 0)
        n = accepted[b] = len(path) - 1
        nodes[b, :n + 1] = path
        out[b, :n] = [tokens[b][t] for t in path[1:]]
        out[b, n] = int(torch.searchsorted(total, final[b] * total[-1], right=True))
    i32 = torch.int32
    return {"accepted": torch.tensor(accepted, dtype=i32), "nodes": torch.tensor(nodes, dtype=i32),
            "tokens": torch.tensor(out, dtype=i32)}


def _exact_move(s):
    c = s["case"]
    r = {}
    for name in ("k", "v"):
        x = s[name].clone()
        flat = x.view(c["layers"], -1, x[0, 0].numel() if c["what"] == "pages" else c["H_kv"] * c["D"])
        old = s[name].view(flat.shape)
        for i, j in zip(s["src"].tolist(), s["dst"].tolist()):
            flat[:, j] = old[:, i]
        r[name] = x
    if c["what"] == "compact":
        r["lengths"] = s["lengths"] + s["accepted"] + 1
    return r
