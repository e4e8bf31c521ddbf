"""What is measured of the operators around a verification step: the cases, their inputs, their
plain forms in elementary torch operations and the calls a serving loop makes of the library.

A request's way through the paged cache: `resize` (pages for the tokens to come, or given back, with
positions and slots of new tokens), `rotate` (norms and position rotation of queries and keys, keys
and values into their slots), `attention` (a chunk of new tokens against all that is cached up to
each of them), `fork` (a request continued several times over shared pages); and, in front of the
verification, `penalize` (repetition, presence and frequency penalties, biases and grammar masks on
the logits of every drafted node). New tokens of all requests are packed: request b has rows
start[b] to start[b + 1].
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one reply, one token at a time: the shortest call, where latency counts
        {"name": "attention single token", "op": "attention", "B": 1, "N": 1, "mix": "whole", "low": 500, "high": 500,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "layout": "token", "dtype": "bf16"},
        # a serving batch: a few prompts' chunks among requests that decode, an odd model of 7 query heads a group
        {"name": "attention mixed batch", "op": "attention", "B": 24, "N": 701, "mix": "mixed", "low": 0, "high": 6011,
         "Hq": 21, "Hkv": 3, "D": 80, "page": 16, "layout": "head", "dtype": "f16"},
        # a whole prompt at once, where the matrix products are all that counts
        {"name": "attention prompt", "op": "attention", "B": 1, "N": 8192, "mix": "whole", "low": 0, "high": 0,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "layout": "token", "dtype": "bf16"},
        # two long documents with a question behind each: some rows over a long axis
        {"name": "attention long", "op": "attention", "B": 2, "N": 137, "mix": "whole", "low": 100003, "high": 131072,
         "Hq": 28, "Hkv": 4, "D": 128, "page": 128, "layout": "token", "dtype": "bf16"},
        # a chain of eight drafted tokens (keys stay outside the cache), and a prompt's far chunk into its pages
        {"name": "rotate nodes", "op": "rotate", "T": 9, "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "norm": True,
         "interleaved": False, "cached": False, "first": 2001, "page": 16, "layout": "token", "dtype": "bf16"},
        {"name": "rotate prompt", "op": "rotate", "T": 8192, "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "norm": True,
         "interleaved": False, "cached": True, "first": 122880, "page": 64, "layout": "token", "dtype": "bf16"},
        # one reply's next token; the benchmark's headline shape with biases and a grammar
        {"name": "penalize single token", "op": "penalize", "B": 1, "N": 1, "tree": "chain", "V": 32000, "low": 700,
         "high": 700, "bias": 0, "mask": False, "dtype": "f32"},
        {"name": "penalize chains", "op": "penalize", "B": 64, "N": 9, "tree": "chain", "V": 128256, "low": 301,
         "high": 8011, "bias": 64, "mask": True, "dtype": "bf16"},
        # pages for one prompt; a batch where some begin, some go on and some have ended
        {"name": "resize single", "op": "resize", "B": 1, "N": 2048, "low": 0, "high": 0, "page": 16, "shared": False},
        {"name": "resize batch", "op": "resize", "B": 512, "N": 600, "low": 17, "high": 8192, "page": 16, "shared": True},
        # four replies to one prompt; a batch of 16 prompts with four replies each
        {"name": "fork single", "op": "fork", "B": 5, "sources": 1, "low": 777, "high": 777, "layers": 4, "H": 8, "D": 128,
         "page": 16, "layout": "token", "dtype": "bf16"},
        {"name": "fork batch", "op": "fork", "B": 80, "sources": 16, "low": 5, "high": 700, "layers": 32, "H": 8, "D": 128,
         "page": 32, "layout": "head", "dtype": "bf16"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "rotate", "rotate", "penalize", "penalize", "resize", "fork"])
    if op == "attention":
        Hq, Hkv = rng.choice([(32, 8), (28, 4), (16, 16), (64, 8), (21, 3), (8, 1), (40, 8)])
        c = {"op": op, "B": _spread(rng, 1, 64), "mix": rng.choice(["whole", "mixed"]), "Hq": Hq, "Hkv": Hkv,
             "D": rng.choice([64, 80, 128, 128, 256]), "page": rng.choice([16, 32, 64, 128]),
             "layout": rng.choice(["token", "head"]), "dtype": rng.choice(["bf16", "f16"])}
        c["N"] = _spread(rng, 1, max(2, min(8192, int(5e8 / (c["B"] * Hq * c["D"])))))
        # as long as the cost allows: no more scores and cached values than the largest listed cases have
        most = min(131072, int(2e8 / (c["B"] * Hkv * c["D"])), int(2.5e11 / (2 * c["B"] * c["N"] * Hq * c["D"]))) - c["N"]
        c["high"] = _spread(rng, 1, max(2, most))
        c["low"] = rng.randint(0, c["high"])
        return c
    if op == "rotate":
        Hq, Hkv = rng.choice([(32, 8), (28, 4), (16, 16), (64, 8), (21, 3), (8, 1)])
        D = rng.choice([64, 80, 128, 128, 256])
        T = _spread(rng, 1, max(2, int(8192 * 48 * 128 / ((Hq + 2 * Hkv) * D))))
        return {"op": op, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "R": rng.choice([D, D, D // 2, 20]), "norm": rng.random() < 0.6,
                "interleaved": rng.random() < 0.3, "cached": rng.random() < 0.5, "first": rng.randint(0, 131072),
                "page": rng.choice([16, 32, 64]), "layout": rng.choice(["token", "head"]),
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]) if T < 4000 else rng.choice(["bf16", "f16"])}
    if op == "penalize":
        V = _spread(rng, 300, 151936)
        B = _spread(rng, 1, 64)
        high = _spread(rng, 2, 8192)
        return {"op": op, "B": B, "N": min(_spread(rng, 1, 64), max(1, int(288 * 128256 / (B * V)))),
                "tree": rng.choice(["chain", "branches", "bushy"]), "V": V, "low": rng.randint(0, high), "high": high,
                "bias": rng.choice([0, 1, 64, 300]), "mask": rng.random() < 0.5, "dtype": rng.choice(["f32", "bf16"])}
    if op == "resize":
        high = _spread(rng, 2, 8192)
        return {"op": op, "B": _spread(rng, 1, 512), "N": _spread(rng, 1, 600), "low": rng.randint(0, high), "high": high,
                "page": rng.choice([16, 32, 64]), "shared": rng.random() < 0.5}
    high = _spread(rng, 2, 700)
    sources = _spread(rng, 1, 16)
    return {"op": op, "B": sources + _spread(rng, 1, 64), "sources": sources, "low": rng.randint(0, high), "high": high,
            "layers": rng.randint(1, 24), "H": rng.choice([1, 4, 8]), "D": rng.choice([64, 80, 128]),
            "page": rng.choice([16, 32]), "layout": rng.choice(["token", "head"]), "dtype": rng.choice(["bf16", "f16"])}


def _parents(kind, n):
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "branches":  # four chains from the root
        return [-1 if i == 0 else 0 if i <= 4 else i - 4 for i in range(n)]
    return [-1 if i == 0 else (i - 1) // 3 for i in range(n)]


def _lengths(c, B=None):
    """Tokens in the cache of each request: from just begun to the longest, in no order."""
    B = B or c["B"]
    if B == 1:
        return [c["high"]]
    at = [(b * 0.6180339887498949) % 1.0 for b in range(B)]
    return [c["low"] + int(round((c["high"] - c["low"]) * (x / max(at)))) for x in at]


def _new(c):
    """New tokens of each request: a chunk each with some of them shorter, a chunk among single tokens, or the
    nodes of a drafted tree (fewer where drafting stopped early)."""
    B, N = c["B"], c["N"]
    if c["op"] == "attention" and c["mix"] == "mixed":
        return [N if b % 8 == 0 else 1 for b in range(B)]
    if c["op"] == "resize":  # every fourth request has ended, some go on by a token, some with a chunk
        return [N if B == 1 else 0 if b % 4 == 3 else 1 if b % 4 == 1 else 1 + (b * 7919) % N for b in range(B)]
    return [N if b % 4 != 3 else 1 + (b * 7919) % N for b in range(B)]


def work(c):
    size = 4 if c.get("dtype") == "f32" else 2
    if c["op"] == "attention":
        n, old = _new(c), _lengths(c)
        T, keys = sum(n), sum(n) + sum(old)
        cells = sum(m * a + m * (m + 1) // 2 for m, a in zip(n, old))
        return {"bytes": size * (2 * keys * c["Hkv"] * c["D"] + 2 * T * c["Hq"] * c["D"]) + 4 * T * c["Hq"],
                "flops": 4 * cells * c["Hq"] * c["D"]}
    if c["op"] == "rotate":
        heads = c["Hq"] + c["Hkv"]
        return {"bytes": 2 * size * c["T"] * (heads + (c["Hkv"] if c["cached"] else 0)) * c["D"] + 4 * c["T"],
                "flops": 8 * c["T"] * heads * c["D"]}
    if c["op"] == "penalize":
        T = sum(_new(c))
        return {"bytes": 2 * size * T * c["V"] + 4 * sum(_lengths(c)) + (T * c["V"] // 8 if c["mask"] else 0) + 8 * c["B"] * c["bias"],
                "flops": 3 * T * c["V"]}
    if c["op"] == "resize":
        n, old = _new(c), _lengths(c)
        pages = sum(-(-(a + m) // c["page"]) for a, m in zip(old, n))
        return {"bytes": 12 * sum(n) + 8 * pages + 16 * c["B"], "flops": 0}
    old, forks = _lengths(c, c["sources"]), c["B"] - c["sources"]
    part = sum(old[j % c["sources"]] % c["page"] for j in range(forks))
    return {"bytes": 4 * size * part * c["layers"] * c["H"] * c["D"] + 8 * sum(-(-old[j % c["sources"]] // c["page"]) for j in range(forks)) + 24 * c["B"],
            "flops": 0}


# --------------------------------------------------------------------------- inputs
def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _cache_view(t, layout):
    """[..., pages, page, heads, width] of storage that is token-major or head-major within a page."""
    return t if layout == "token" else t.transpose(-3, -2)


def _caches(lead, total, c, heads, g):
    shape = (total, c["page"], heads, c["D"]) if c["layout"] == "token" else (total, heads, c["page"], c["D"])
    return [_cache_view(torch.randn(lead + shape, dtype=DTYPES[c["dtype"]], device="cuda", generator=g), c["layout"]) for _ in range(2)]


def _starts(n):
    start = [0]
    for m in n:
        start.append(start[-1] + m)
    return start


def _table(rows, width):
    return _ints([r + [-1] * (width - len(r)) for r in rows])


def prepare(case, seed):
    c, rng = case, random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"attention": _prepare_attention, "rotate": _prepare_rotate, "penalize": _prepare_penalize,
            "resize": _prepare_resize, "fork": _prepare_fork}[c["op"]](c, rng, g)


def _prepare_attention(c, rng, g):
    n, old = _new(c), _lengths(c)
    T, page = sum(n), c["page"]
    owned = [-(-(a + m) // page) for a, m in zip(old, n)]
    ids = list(range(sum(owned) + 3))
    rng.shuffle(ids)
    at = _starts(owned)
    k, v = _caches((), len(ids), c, c["Hkv"], g)
    # what the projection before it gives: queries, keys and values of a token side by side
    qkv = torch.randn((T, c["Hq"] + 2 * c["Hkv"], c["D"]), dtype=DTYPES[c["dtype"]], device="cuda", generator=g)
    q = qkv[:, :c["Hq"]]
    q.mul_(1.5)  # some rows with one strong key, as in a model
    return {"case": dict(c), "T": T, "max_chunk": max(n), "q": q, "k_cache": k, "v_cache": v,
            "block_table": _table([ids[a:b] for a, b in zip(at, at[1:])], max(owned)), "prefix_len": _ints(old),
            "chunk_start": _ints(_starts(n)), "out": torch.empty((T, c["Hq"], c["D"]), dtype=q.dtype, device="cuda")}


def _prepare_rotate(c, rng, g):
    T, Hq, Hkv, D, dt = c["T"], c["Hq"], c["Hkv"], c["D"], DTYPES[c["dtype"]]
    qkv = torch.randn((T, Hq + 2 * Hkv, D), dtype=dt, device="cuda", generator=g)
    q, k, v = qkv.split([Hq, Hkv, Hkv], dim=1)
    q.mul_(3.0)
    half = c["R"] // 2
    s = {"case": dict(c), "q": q, "k": k, "v": v,
         "position": c["first"] + torch.arange(T, device="cuda", dtype=torch.int32),
         "inv_freq": (500000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda(),
         "q_weight": None, "k_weight": None, "out_q": torch.empty((T, Hq, D), dtype=dt, device="cuda")}
    if c["norm"]:
        s["q_weight"], s["k_weight"] = (1 + 0.2 * torch.randn(2, D, device="cuda", generator=g)).to(dt)
    if c["cached"]:
        page, off = c["page"], c["first"] % c["page"]
        ids = list(range(-(-(off + T) // page) + 2))
        rng.shuffle(ids)
        at = off + torch.arange(T, device="cuda")
        s["slots"] = _ints(ids, torch.int64)[at // page] * page + at % page
        s["k_cache"], s["v_cache"] = _caches((), len(ids), c, Hkv, g)
    else:
        s["out_k"] = torch.empty((T, Hkv, D), dtype=dt, device="cuda")
    return s


def _prepare_penalize(c, rng, g):
    n, old, B, V, N = _new(c), _lengths(c), c["B"], c["V"], c["N"]
    T = sum(n)

    def words(*shape):  # tokens as often as in text: rank r about 1 / r of the time, ranks in no order of ids
        rank = (V ** torch.rand(shape, device="cuda", generator=g, dtype=torch.float64)).long().clamp(1, V) - 1
        return (rank * 7919 % V).int()

    s = {"case": dict(c), "T": T, "max_nodes": N, "node_start": _ints(_starts(n)), "tokens": words(T),
         "logits": (4.0 * torch.randn((T, V), device="cuda", generator=g)).to(DTYPES[c["dtype"]]),
         "history": words(B, max(1, max(old))), "prefix_len": _ints(old), "prompt_len": _ints([a // 2 for a in old]),
         "repetition": 1.0 + 0.3 * torch.rand(B, device="cuda", generator=g),
         "presence": 0.5 * torch.rand(B, device="cuda", generator=g), "frequency": 0.3 * torch.rand(B, device="cuda", generator=g),
         "ancestors": None, "bias_start": None, "bias_token": None, "bias": None, "mask": None}
    # what a request generates repeats what it has seen: some drafted tokens are of its history
    if max(old) > 0:
        b = torch.repeat_interleave(torch.arange(B, device="cuda"), _ints(n).long())
        seen = s["history"][b, (torch.rand(T, device="cuda", generator=g) * s["prefix_len"][b]).long()]
        s["tokens"] = torch.where((torch.rand(T, device="cuda", generator=g) < 0.5) & (s["prefix_len"][b] > 0), seen, s["tokens"])
    if c["tree"] != "chain":
        up = [p for m in n for p in _parents(c["tree"], m)]
        bits = []
        for lo, m in zip(_starts(n), n):
            own_bits = []
            for i in range(m):
                own_bits.append((own_bits[up[lo + i]] if up[lo + i] >= 0 else 0) | 1 << i)
            bits += own_bits
        W = (N + 63) // 64
        s["ancestors"] = _ints([[(x >> 64 * w & (1 << 64) - 1) - ((x >> 64 * w + 63 & 1) << 64) for w in range(W)] for x in bits], torch.int64)
    if c["bias"]:
        k = c["bias"]
        s["bias_start"] = _ints([k * b for b in range(B + 1)])
        s["bias_token"] = torch.randint(0, V, (k * B,), device="cuda", generator=g, dtype=torch.int32)
        s["bias"] = 2.0 * torch.randn(k * B, device="cuda", generator=g)
    if c["mask"]:  # a grammar that leaves about half of the ids
        s["mask"] = torch.randint(-2 ** 31, 2 ** 31, (T, (V + 31) // 32), device="cuda", generator=g, dtype=torch.int64).int()
    s["out"] = torch.empty_like(s["logits"])
    return s


def _prepare_resize(c, rng, g):
    n, old, B, page = _new(c), _lengths(c), c["B"], c["page"]
    held = [-(-a // page) for a in old]  # pages of what is cached
    # requests end (every fourth), and some were given room for drafts that were not accepted
    old = [0 if B > 1 and b % 4 == 3 else a for b, a in enumerate(old)]
    held = [k + (1 if b % 8 == 1 else 0) for b, k in enumerate(held)]
    ids = list(range(sum(held) + sum(-(-m // page) + 1 for m in n)))
    rng.shuffle(ids)
    at = _starts(held)
    rows = [ids[a:b] for a, b in zip(at, at[1:])]
    shares = [0] * len(ids)
    if c["shared"]:  # some requests began as a fork of the one before
        for b in range(1, B):
            if b % 3 == 2:
                for j in range(min(len(rows[b]), len(rows[b - 1]), 1 + b % 64)):
                    rows[b][j] = rows[b - 1][j]
                    shares[rows[b][j]] += 1
    used = set(p for r in rows for p in r)
    free = [p for p in ids if p not in used]
    width = max(-(-(a + m) // page) for a, m in zip(old, n))
    return {"case": dict(c), "T": sum(n), "num_pages": len(ids), "prefix_len": _ints(old), "pages": _ints(held),
            "block_table": _table(rows, max(width, max(held))), "free_pages": _ints([-1] * (len(ids) - len(free)) + free),
            "free_head": _ints([len(ids) - len(free)]), "chunk_start": _ints(_starts(n)),
            "shares": _ints(shares) if c["shared"] else None}


def _prepare_fork(c, rng, g):
    S, B, page = c["sources"], c["B"], c["page"]
    old = _lengths(c, S)
    held = [-(-a // page) for a in old]
    ids = list(range(sum(held) + B - S + 2))
    rng.shuffle(ids)
    at = _starts(held)
    rows = [ids[a:b] for a, b in zip(at, at[1:])] + [[] for _ in range(B - S)]
    k, v = _caches((c["layers"],), len(ids), c, c["H"], g)
    to = list(range(S, B))
    return {"case": dict(c), "source": _ints([(t - S) % S for t in to]), "target": _ints(to),
            "prefix_len": _ints(old + [0] * (B - S)), "pages": _ints(held + [0] * (B - S)),
            "block_table": _table(rows, max(held) + 1), "free_pages": _ints(ids), "free_head": _ints([sum(held)]),
            "shares": _ints([0] * len(ids)), "num_pages": len(ids), "k_cache": k, "v_cache": v}


# --------------------------------------------------------------------------- one pass
def run(s):
    return {"attention": _attention, "rotate": _rotate, "penalize": _penalize, "resize": _resize, "fork": _fork}[s["case"]["op"]](s)


def _rows(start, T, N):
    """The packed rows' requests and places: request [T], index in the request [T], counts [B], and the
    packed row of (request, index) clamped to a row that exists [B, N]."""
    n = (start[1:] - start[:-1]).long()
    first = start[:-1].long()
    b = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n, output_size=T)
    i = torch.arange(T, device=n.device) - first[b]
    at = (first[:, None] + torch.arange(N, device=n.device)).clamp(max=T - 1)
    return b, i, n, at


def _attention(s):
    c = s["case"]
    if own:
        from device_draft_verification_specverify_amd import serving
        return list(serving.specverify_chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["prefix_len"],
                                                       s["chunk_start"], max_chunk=s["max_chunk"], out=s["out"], want_lse=True))
    T, N, B, D, Hkv = s["T"], s["max_chunk"], c["B"], c["D"], c["Hkv"]
    G = c["Hq"] // Hkv
    b, i, n, at = _rows(s["chunk_start"], T, N)
    table = s["block_table"].long().clamp(min=0)
    L = table.shape[1] * c["page"]

    def keys(cache):  # [B, Hkv, L, D] in 32 bits
        return cache[table].float().flatten(1, 2).transpose(1, 2)

    last = s["prefix_len"].long()[:, None] + torch.arange(N, device=table.device)  # [B, N]
    seen = (torch.arange(L, device=table.device) <= last[:, :, None])[:, None, None]
    q = s["q"][at].float().view(B, N, Hkv, G, D).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(q.reshape(B, Hkv, G * N, D), keys(s["k_cache"]).transpose(2, 3).contiguous())
    scores = scores.view(B, Hkv, G, N, L).mul_(D ** -0.5).masked_fill_(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    scores = scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    # (pages behind a request's last hold another one's values: finite, and of weight zero)
    out = torch.matmul(scores.view(B, Hkv, G * N, L), keys(s["v_cache"]).contiguous()).view(B, Hkv, G, N, D)
    out = (out / total).permute(0, 3, 1, 2, 4).reshape(B, N, c["Hq"], D)[b, i].to(s["q"].dtype)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, N, c["Hq"])[b, i]
    return [out, lse]


def _rotate(s):
    c = s["case"]
    if own:
        from device_draft_verification_specverify_amd import serving
        if c["cached"]:
            q, _ = serving.specverify_rotate(s["q"], s["k"], s["v"], s["position"], s["inv_freq"], q_weight=s["q_weight"],
                                             k_weight=s["k_weight"], eps=1e-6, interleaved=c["interleaved"], out_q=s["out_q"],
                                             slots=s["slots"], k_cache=s["k_cache"], v_cache=s["v_cache"])
            return [q, s["k_cache"], s["v_cache"]]
        return list(serving.specverify_rotate(s["q"], s["k"], None, s["position"], s["inv_freq"], q_weight=s["q_weight"],
                                              k_weight=s["k_weight"], eps=1e-6, interleaved=c["interleaved"], out_q=s["out_q"],
                                              out_k=s["out_k"]))
    half = c["R"] // 2
    angle = s["position"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
        r = x[..., :2 * half]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([r, x[..., 2 * half:]], -1).to(s["q"].dtype)

    q, k = turned(s["q"], s["q_weight"]), turned(s["k"], s["k_weight"])
    if not c["cached"]:
        return [q, k]
    page, off = s["slots"] // c["page"], s["slots"] % c["page"]
    s["k_cache"][page, off] = k
    s["v_cache"][page, off] = s["v"]
    return [q, s["k_cache"], s["v_cache"]]


def _penalize(s):
    c = s["case"]
    if own:
        from device_draft_verification_specverify_amd import serving
        return serving.specverify_penalize(s["logits"], s["tokens"], s["node_start"], s["history"], s["prefix_len"], s["prompt_len"],
                                           s["repetition"], s["presence"], s["frequency"], ancestors=s["ancestors"],
                                           max_nodes=s["max_nodes"], bias_start=s["bias_start"], bias_token=s["bias_token"],
                                           bias=s["bias"], mask=s["mask"], out=s["out"])
    T, N, B, V = s["T"], s["max_nodes"], c["B"], c["V"]
    b, i, n, at = _rows(s["node_start"], T, N)
    idx = torch.arange(N, device=n.device)
    if s["ancestors"] is None:
        up = idx <= i[:, None]
    else:
        up = (s["ancestors"][:, idx // 64] >> (idx % 64)) & 1 > 0
    up = up & (idx < n[b][:, None])  # [T, N]
    j = torch.arange(s["history"].shape[1], device=n.device)
    kept, made = j < s["prompt_len"][:, None], (j < s["prefix_len"][:, None]) & (j >= s["prompt_len"][:, None])
    seen = torch.zeros((B, V), device=n.device).scatter_add_(1, s["history"].long(), kept.float())[b]
    count = torch.zeros((B, V), device=n.device).scatter_add_(1, s["history"].long(), made.float())[b]
    count.scatter_add_(1, s["tokens"][at[b]].long(), up.float())
    x = s["logits"].float()
    rep = s["repetition"][b][:, None]
    x = torch.where(seen + count > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = torch.where(count > 0, x - (s["frequency"][b][:, None] * count + s["presence"][b][:, None]), x)
    if s["bias"] is not None:
        whose = torch.arange(B, device=n.device).repeat_interleave(c["bias"])
        x += torch.zeros((B, V), device=n.device).index_put_((whose, s["bias_token"].long()), s["bias"], accumulate=True)[b]
    if s["mask"] is not None:
        v = torch.arange(V, device=n.device)
        x = torch.where((s["mask"][:, v // 32] >> (v % 32)) & 1 > 0, x, float("-inf"))
    return x.to(s["logits"].dtype)


def _resize(s):
    c, page, T = s["case"], s["case"]["page"], s["T"]
    if own:
        from device_draft_verification_specverify_amd import serving
        o = serving.specverify_pages_resize(s["prefix_len"], s["pages"], s["block_table"], s["free_pages"], s["free_head"],
                                            page_size=page, num_pages=s["num_pages"], chunk_start=s["chunk_start"], rows=T,
                                            shares=s["shares"])
        return [o.pages, o.free_head, o.shares, o.position, o.slots, s["block_table"], s["free_pages"]]
    start, table, free = s["chunk_start"].long(), s["block_table"], s["free_pages"]
    n, length, pages, head = start[1:] - start[:-1], s["prefix_len"].long(), s["pages"].long(), s["free_head"].long()
    need = (length + n + page - 1) // page
    j = torch.arange(table.shape[1], device=table.device)
    # what is given back, and what of it nobody holds any more, by id
    back = (j >= need[:, None]) & (j < pages[:, None])
    given = torch.zeros(s["num_pages"] + 1, dtype=torch.int64, device=table.device)
    given.scatter_add_(0, torch.where(back, table.long(), s["num_pages"]).flatten(), back.long().flatten())
    given = given[:-1]
    shares = s["shares"].long() if s["shares"] is not None else torch.zeros_like(given)
    freed = given > shares
    head = head - freed.sum()
    place = torch.where(freed, head + freed.cumsum(0) - 1, free.numel())
    free = torch.cat([free, free[:1]]).scatter(0, place, torch.arange(s["num_pages"], device=table.device, dtype=torch.int32))[:-1]
    # what is taken, in order of requests
    more = (need - pages).clamp(min=0)
    before = more.cumsum(0) - more
    fits = (more == 0) | (before + more <= free.numel() - head)
    more = torch.where(fits, more, 0)
    new = (j >= pages[:, None]) & (j < (pages + more)[:, None])
    grown = torch.where(new, free[(head + before[:, None] + j - pages[:, None]).clamp(0, free.numel() - 1)], table)
    b = torch.repeat_interleave(torch.arange(n.numel(), device=table.device), n, output_size=T)
    to = length[b] + torch.arange(T, device=table.device) - start[b]
    slots = torch.where(fits[b], grown[b, to // page].long() * page + to % page, -1)
    return [torch.where(pages > need, need, pages + more).int(), (head + more.sum()).int(),
            (shares - given).clamp(min=0).int() if s["shares"] is not None else None, to.int(), slots, grown, free]


def _fork(s):
    c, page = s["case"], s["case"]["page"]
    if own:
        from device_draft_verification_specverify_amd import serving
        o = serving.specverify_pages_fork(s["source"], s["target"], s["prefix_len"], s["pages"], s["block_table"], s["free_pages"],
                                          s["free_head"], s["shares"], s["k_cache"], s["v_cache"])
        return [o.prefix_len, o.pages, o.free_head, o.shares, s["block_table"], s["k_cache"], s["v_cache"]]
    source, target, table = s["source"].long(), s["target"].long(), s["block_table"]
    length = s["prefix_len"].long()[source]
    full, part = length // page, length % page
    takes = (part > 0).long()
    before = takes.cumsum(0) - takes
    fits = (takes == 0) | (before + takes <= s["free_pages"].numel() - s["free_head"].long())
    new = s["free_pages"][(s["free_head"].long() + before).clamp(max=s["free_pages"].numel() - 1)].long()
    j = torch.arange(table.shape[1], device=table.device)
    rows = table[source]
    shared = (j < full[:, None]) & fits[:, None]
    row = torch.where(shared, rows, table[target])
    row = torch.where((j == full[:, None]) & ((takes > 0) & fits)[:, None], new[:, None].int(), row)
    grown = table.index_copy(0, target, row)
    shares = torch.cat([s["shares"], s["shares"][:1]]).scatter_add(
        0, torch.where(shared, rows.long(), s["num_pages"]).flatten(), shared.int().flatten())[:-1]
    # the tokens of the last page that is not full; a place that takes nothing takes itself
    old = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None]).long().clamp(min=0).expand(-1, page)
    off = torch.arange(page, device=table.device).expand_as(old)
    to = torch.where((off < part[:, None]) & fits[:, None], new[:, None], old)
    for cache in (s["k_cache"], s["v_cache"]):
        cache[:, to, off] = cache[:, old, off]
    done = torch.where(fits, length, s["prefix_len"].long()[target]).int()
    owned = torch.where(fits, full + takes, s["pages"].long()[target]).int()
    return [s["prefix_len"].index_copy(0, target, done), s["pages"].index_copy(0, target, owned),
            (s["free_head"] + (takes * fits).sum()).int(), shares, grown, s["k_cache"], s["v_cache"]]


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    c = case
    if c["op"] in ("resize", "fork"):  # whole numbers and copies: equal or not
        return None
    s = prepare(case, seed)
    return {"attention": _exact_attention, "rotate": _exact_rotate, "penalize": _exact_penalize}[c["op"]](c, s)


def _exact_attention(c, s):
    D, G, page = c["D"], c["Hq"] // c["Hkv"], c["page"]
    start, old = s["chunk_start"].tolist(), s["prefix_len"].tolist()
    out = torch.empty((s["T"], c["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["T"], c["Hq"]), dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        lo, hi = start[b], start[b + 1]
        end = old[b] + hi - lo
        ids = s["block_table"][b][:-(-end // page)].long()
        for h in range(c["Hkv"]):
            k, v = (s[x + "_cache"][ids, :, h].reshape(-1, D)[:end].double() for x in "kv")
            for a in range(lo, hi, 1024):  # rows at a time
                z = min(a + 1024, hi)
                sees = torch.arange(old[b] + a - lo + 1, old[b] + z - lo + 1, device="cuda")
                q = s["q"][a:z, h * G:(h + 1) * G].double().reshape(-1, D)
                t = (q @ k.T.contiguous() / math.sqrt(D)).view(z - a, G, end)
                t.masked_fill_((torch.arange(end, device="cuda") >= sees[:, None])[:, None], float("-inf"))
                one = torch.logsumexp(t, 2)
                lse[a:z, h * G:(h + 1) * G] = one
                out[a:z, h * G:(h + 1) * G] = (torch.exp(t - one[:, :, None]).view((z - a) * G, end) @ v).view(z - a, G, D)
    return [out, lse]


def _exact_rotate(c, s):
    half, page = c["R"] // 2, c["page"]
    turn = torch.polar(torch.ones((c["T"], half), dtype=torch.float64, device="cuda"),
                       torch.outer(s["position"].double(), s["inv_freq"].double()))
    one = torch.arange(half, device="cuda")
    first, second = (2 * one, 2 * one + 1) if c["interleaved"] else (one, one + half)

    def turned(x, weight):
        y = x.double().clone()
        if weight is not None:
            y = y / ((y * y).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * weight.double()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k = turned(s["q"], s["q_weight"]), turned(s["k"], s["k_weight"])
    if not c["cached"]:
        return [q, k]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc.index_put_((s["slots"] // page, s["slots"] % page), k)
    vc.index_put_((s["slots"] // page, s["slots"] % page), s["v"].double())
    return [q, kc, vc]


def _exact_penalize(c, s):
    V, start = c["V"], s["node_start"].tolist()
    out = s["logits"].double()
    for b, (old, prompt) in enumerate(zip(s["prefix_len"].tolist(), s["prompt_len"].tolist())):
        told = torch.bincount(s["history"][b, :prompt].long(), minlength=V)
        said = torch.bincount(s["history"][b, prompt:old].long(), minlength=V)
        rep, pres, freq = (s[x][b].double() for x in ("repetition", "presence", "frequency"))
        add = torch.zeros(V, dtype=torch.float64, device="cuda")
        if s["bias"] is not None:
            lo, hi = s["bias_start"][b:b + 2].tolist()
            add.index_add_(0, s["bias_token"][lo:hi].long(), s["bias"][lo:hi].double())
        tokens = s["tokens"][start[b]:start[b + 1]].long()
        for i in range(len(tokens)):
            if s["ancestors"] is None:
                line = tokens[:i + 1]
            else:
                words = [w & (1 << 64) - 1 for w in s["ancestors"][start[b] + i].tolist()]
                line = tokens[[m for m in range(len(tokens)) if words[m // 64] >> (m % 64) & 1]]
            times = said + torch.bincount(line, minlength=V)
            x = out[start[b] + i]
            x = torch.where((told + times) > 0, torch.where(x < 0, x * rep, x / rep), x)
            x = x - times * freq - (times > 0) * pres + add
            if s["mask"] is not None:
                keep = (s["mask"][start[b] + i][:, None] >> torch.arange(32, device="cuda")) & 1
                x[keep.flatten()[:V] == 0] = -math.inf
            out[start[b] + i] = x
    return out
