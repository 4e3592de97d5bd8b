"""Measured cases of a video transformer block's step over a paged cache: the norms
between two blocks with gate, residual scale and modulation (``residual_norm``), the
cache write with positions of three axes, the write into an 8-bit cache with a scale
for each block of 16 tokens and head, and the attention over that cache.

Each case runs either in its plain form (elementary torch operations in 32 bits,
angles in 64) or, with ``own`` set, through the package's calls.  Both forms take what
``prepare`` makes.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 16            # tokens that share a scale
HEADS = [(10, 10), (40, 40), (32, 8), (40, 8), (16, 2), (12, 4), (20, 4), (7, 1)]


# ---------------------------------------------------------------- the cases
def listed():
    norm = dict(op="norm", mods="fp32", post="none", gate=True)
    write = dict(op="write", pad=0, norm=True, axes="", t_pairs=0, y_pairs=0)
    att = dict(op="attention", causal=True, window=0)
    return [
        # a few decoding tokens between two blocks: latency
        dict(norm, name="norm_tokens", tokens=9, width=1280, stream="bf16", kind="rms", rows=1, mods="bf16"),
        # one video frame between attention and the feed-forward part, the stream kept in 32 bits, one time step
        dict(norm, name="norm_frame", tokens=757, width=5120, stream="fp32", kind="layer", rows=1),
        # the frames of several sessions at time steps of their own, with a norm behind the block as well
        dict(norm, name="norm_sessions", tokens=16384, width=5120, stream="bf16", kind="rms", rows=16, post="rms"),
        # one frame's queries, keys and values, turned by (t, y, x), into the cache with a scale per head
        dict(write, name="axes_frame", tokens=757, requests=1, before=1217, q_heads=40, kv_heads=40, dim=128, cache="e4m3",
             pairing="adjacent", page=64, axes="section", t_pairs=22, y_pairs=21, lens=1),
        # images and text of several requests, shared key/value heads, the frequencies of the whole head, padded
        dict(write, name="axes_images", tokens=12001, requests=7, before=3000, q_heads=32, kv_heads=8, dim=128, cache="bf16",
             pairing="halves", page=64, axes="head", t_pairs=16, y_pairs=24, lens=2, pad=63),
        # one token for each of a batch, into blocks that hold some already
        dict(write, name="blocks_decode", tokens=48, requests=48, before=300, q_heads=10, kv_heads=10, dim=128,
             cache="blocks", pairing="adjacent", page=64, lens=3),
        # one frame, (t, y, x), block scales
        dict(write, name="blocks_frame", tokens=757, requests=1, before=1217, q_heads=40, kv_heads=40, dim=128,
             cache="blocks", pairing="adjacent", page=64, axes="section", t_pairs=22, y_pairs=21, lens=4),
        # prompts of several requests, shared key/value heads
        dict(write, name="blocks_prompts", tokens=16384, requests=5, before=2000, q_heads=32, kv_heads=8, dim=128,
             cache="blocks", pairing="halves", page=64, lens=5),
        # a single request that decodes early in its life: latency
        dict(att, name="decode_one", requests=1, new=1, long=700, q_heads=32, kv_heads=8, dim=128, page=64, lens=6),
        # a full batch of decoding requests of ragged lengths
        dict(att, name="decode_batch", requests=128, new=1, long=16384, q_heads=32, kv_heads=8, dim=128, page=64, lens=7),
        # one frame over the filled window, every token sees every other
        dict(att, name="frame", requests=1, new=757, long=5788, q_heads=40, kv_heads=40, dim=128, page=64, lens=8,
             causal=False),
        # a chunk of a long prompt behind what is cached
        dict(att, name="chunk", requests=1, new=4096, long=16384, q_heads=32, kv_heads=8, dim=128, page=64, lens=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "write", "write", "attention", "attention"])
    if kind == "norm":
        width = 8 * _log(rng, 8, 1024)
        tokens = _log(rng, 1, min(16384, 16384 * 5120 // width))
        return dict(op="norm", tokens=tokens, width=width, stream=rng.choice(["bf16", "fp32"]),
                    kind=rng.choice(["rms", "layer"]), post=rng.choice(["none", "none", "rms", "layer"]),
                    gate=rng.random() < 0.75, mods=rng.choice(["bf16", "fp32"]),
                    rows=rng.choice([1, min(tokens, 5), min(tokens, 37)]))
    dim = rng.choice([64, 128, 128])
    qh, kh = rng.choice([h for h in HEADS if (h[0] + 2 * h[1]) * dim <= 120 * 128])
    c = dict(op=kind, q_heads=qh, kv_heads=kh, dim=dim, page=rng.choice([16, 32, 64, 128, 256]), lens=rng.randrange(10 ** 6))
    if kind == "write":
        t = _log(rng, 1, min(16384, 16384 * 48 * 128 // ((qh + 2 * kh) * dim)))
        cache = rng.choice(["blocks", "blocks", "e4m3", "bf16"])
        axes = rng.choice(["section", "head", ""]) if cache == "blocks" else rng.choice(["section", "head"])
        tp = rng.randint(1, dim // 2 - 2) if axes else 0
        yp = rng.randint(0, dim // 2 - 1 - tp) if axes else 0
        return dict(c, tokens=t, requests=rng.choice([1, min(t, 6), min(t, 100)]), before=_log(rng, 16, 4000), cache=cache,
                    axes=axes, t_pairs=tp, y_pairs=yp, pad=rng.choice([0, 0, 13]), norm=rng.random() < 0.75,
                    pairing=rng.choice(["adjacent", "halves"]))
    if rng.random() < 0.5:   # single tokens and drafts
        new = rng.choice([1, 1, 1, 2, 3, 5])
        long = _log(rng, max(8, new), 32000)
        most = max(1, min(128, 128 * 16384 * 8 * 128 // (long * kh * dim), 2 ** 31 // (long * qh * new)))
        return dict(c, requests=_log(rng, 1, most), new=new, long=long, causal=True, window=rng.choice([0, 0, 0, 500]))
    new = _log(rng, 6, 4096)
    full = 26 * 4096 * 16384   # query rows x keys
    long = max(new, min(_log(rng, new, 16384), full // (qh * new)))
    most = max(1, min(16, full // (long * qh * new)))
    causal = rng.random() < 0.75
    return dict(c, requests=_log(rng, 1, most), new=new, long=long, causal=causal,
                window=rng.choice([0, 0, 700]) if causal else 0)


def _lengths(case):
    """(cached before the step, new) of every request, from the case alone."""
    r, n = random.Random(case["lens"]), case["requests"]
    if case["op"] == "write":
        share = [r.random() + 0.1 for _ in range(n)]
        spare = case["tokens"] - n
        new = [1 + int(spare * x / sum(share)) for x in share]
        new[0] += case["tokens"] - sum(new)
        return [case["before"]] + [r.randint(0, case["before"]) for _ in range(n - 1)], new
    new = [case["new"]] + [r.randint(max(1, case["new"] // 2), case["new"]) for _ in range(n - 1)]
    total = [case["long"]] + [_log(r, max(x, case["long"] // 8), max(x, case["long"])) for x in new[1:]]
    return [t - x for t, x in zip(total, new)], new


def _pairs(case, before, new):
    """How many (query, key) pairs of one request the mask leaves, and how many keys it reads."""
    if not case["causal"]:
        return new * (before + new), before + new
    w = case["window"]
    if not w:
        return new * before + new * (new + 1) // 2, before + new
    grow = max(0, min(new, w - before))       # tokens whose window still reaches back to the start
    return grow * before + grow * (grow + 1) // 2 + (new - grow) * w, min(before + new, new - 1 + w)


def work(case):
    if case["op"] == "norm":
        n, d = case["tokens"], case["width"]
        stream, mods = [4 if case[k] == "fp32" else 2 for k in ("stream", "mods")]
        tables = case["rows"] * d * mods * (3 if case["gate"] else 2) + (2 * d if case["post"] != "none" else 0)
        return {"bytes": n * d * (2 * stream + 4) + tables + (4 * n if case["rows"] > 1 else 0),
                "flops": n * d * (10 if case["post"] == "none" else 15)}
    qh, kh, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "write":
        t, size = case["tokens"], 2 if case["cache"] == "bf16" else 1
        where = (12 if case["axes"] else 4) + 4
        return {"bytes": t * d * (2 * (qh + 2 * kh) + 2 * qh + size * 2 * kh) + t * where + 4 * d * t,
                "flops": 8 * t * d * (qh + kh)}
    before, new = _lengths(case)
    both = [_pairs(case, b, n) for b, n in zip(before, new)]
    keys = sum(k for _, k in both)
    return {"bytes": 4 * d * qh * sum(new) + 2 * kh * (d * keys + keys // BLOCK),
            "flops": 4 * d * qh * sum(p for p, _ in both)}


# ---------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _codes(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _type(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _norm_case(case, g):
    n, d, m = case["tokens"], case["width"], case["rows"]
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    # a residual stream: uneven columns, a few large ones, a mean that is not zero
    h = rand(n, d) * (0.5 + 2.0 * torch.rand(d, generator=g, device=DEV)) + 0.3 * rand(d)
    h[:, :: max(1, d // 5)] *= 12.0
    s = dict(h=h.to(_type(case["stream"])), y=rand(n, d).to(torch.bfloat16))
    s["mod"] = (0.4 * rand(m, 3, d)).to(_type(case["mods"]))   # gate, scale, shift, side by side as a projection makes them
    # (a session's tokens lie together)
    s["rows"] = torch.randint(0, m, (n,), generator=g, device=DEV).sort()[0].to(torch.int32) if m > 1 else None
    s["post_w"] = (0.5 + torch.rand(d, generator=g, device=DEV)).to(torch.bfloat16) if case["post"] != "none" else None
    s["h_out"] = torch.zeros_like(s["h"])
    s["x_out"] = torch.zeros((n, d), dtype=torch.bfloat16, device=DEV)
    return s


def _tables(total, page, g, spare):
    """Block tables of requests of the given lengths in a shuffled pool, and the pages left over."""
    need = [-(-t // page) for t in total]
    num = sum(need) + spare
    order = torch.randperm(num, generator=g, device=DEV).to(torch.int32)
    n = torch.tensor(need, device=DEV)
    first = torch.cumsum(n, 0) - n
    w = torch.arange(max(need), device=DEV)
    at = (first[:, None] + w).clamp(max=num - 1)
    table = torch.where(w < n[:, None], order[at], torch.full((), -1, dtype=torch.int32, device=DEV))
    return table.contiguous(), order[sum(need):].contiguous(), num


def _pool(case, num, g):
    shape = (num, case["kv_heads"], case["page"], case["dim"])
    bf16 = case.get("cache") == "bf16"

    def one():
        x = torch.empty(shape, dtype=torch.bfloat16 if bf16 else torch.float8_e4m3fn, device=DEV)
        for i in range(0, num, 4096):   # no 32-bit copy of a whole large pool
            y = torch.randn((min(4096, num - i),) + shape[1:], generator=g, device=DEV)
            x[i:i + 4096] = y.to(torch.bfloat16) if bf16 else _codes(y * 100.0)
        return x

    return one(), one()


def _paged_case(case, g):
    before, new = _lengths(case)
    total = [b + n for b, n in zip(before, new)]
    p, kh, d = case["page"], case["kv_heads"], case["dim"]
    table, free, num = _tables(total, p, g, 5)
    kc, vc = _pool(case, num, g)
    s = dict(table=table, free=free, num=num, kc=kc, vc=vc, before=_ints(before), total=_ints(total), new=_ints(new),
             cu=torch.cumsum(torch.tensor([0] + new, device=DEV), 0).to(torch.int32), most_new=max(new), most_len=max(total))
    if case.get("cache", "blocks") == "blocks":
        # the exponents (biased by 127) of scales that suit the codes and differ from block to block
        shape = (num, kh, p // BLOCK)
        s["ks"], s["vs"] = [(127 + torch.randint(lo, -4, shape, generator=g, device=DEV)).to(torch.uint8) for lo in (-9, -10)]
    elif case["cache"] == "e4m3":
        s["sk"], s["sv"] = [0.005 + 0.01 * torch.rand(kh, generator=g, device=DEV) for _ in range(2)]
    return s


def _attention_case(case, g):
    s = _paged_case(case, g)
    n = int(s["cu"][-1])
    s["q"] = (1.5 * torch.randn((n, case["q_heads"], case["dim"]), generator=g, device=DEV)).to(torch.bfloat16)
    s["out"] = torch.zeros_like(s["q"])
    return s


def _write_case(case, g):
    s = _paged_case(case, g)
    qh, kh, d, p = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    t, cols = case["tokens"], (qh + 2 * kh) * d
    qkv = torch.randn((t + case["pad"], cols), generator=g, device=DEV).to(torch.bfloat16)
    s["qkv"] = qkv * (0.5 + 2.0 * torch.rand((1, cols), generator=g, device=DEV)).to(torch.bfloat16)
    s["q_out"] = torch.zeros((t + case["pad"], qh, d), dtype=torch.bfloat16, device=DEV)
    s["wq"], s["wk"] = [(0.5 + torch.rand(d, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None
                        for _ in range(2)]
    i = torch.arange(t, device=DEV)
    b = torch.searchsorted(s["cu"][1:].long(), i, right=True)
    at = s["before"].long()[b] + i - s["cu"].long()[b]
    s["slots"] = (s["table"].long()[b, at // p] * p + at % p).to(torch.int32)
    # (t, y, x) of a request's tokens: pictures of 28 x 27, one after the other
    s["at"] = at.to(torch.int32)
    s["pos"] = torch.zeros((t + case["pad"], 3), dtype=torch.int32, device=DEV)
    s["pos"][:t] = torch.stack([at // 756, at % 756 // 27, at % 27], -1).to(torch.int32)
    return s


def _case(case, seed):
    """The tensors of a case, the same for every form."""
    g = _gen(seed)
    s = {"norm": _norm_case, "write": _write_case, "attention": _attention_case}[case["op"]](case, g)
    s["case"] = case
    return s


def prepare(case, seed):
    s = _case(case, seed)
    if own and case["op"] != "norm":
        s["pages"] = _pages(s)
    return s


def _pages(s):
    """The cache a program keeps, in the state that the case's tensors describe."""
    from ring_kv_cache_gb300 import KvPages
    c = s["case"]
    rows, width = s["table"].shape
    n, p, blocks = int(s["cu"][-1]), c["page"], c.get("cache", "blocks") == "blocks"
    three = dict(rope3d=(c["t_pairs"], c["y_pairs"]), rope_frequencies=c["axes"], max_position=1024) if c.get("axes") else {}
    pages = KvPages(c["q_heads"], c["kv_heads"], c["dim"], page_size=p, num_pages=s["num"], max_requests=rows,
                    max_request_tokens=width * p, max_tokens=n + c.get("pad", 0),
                    cache_dtype=torch.bfloat16 if c.get("cache") == "bf16" else torch.float8_e4m3fn, block_scales=blocks,
                    rope_pairing=c.get("pairing", "adjacent"), **three)
    # the step's own new pages are the next ones the plan takes: back onto the free list in its order
    used, w = s["table"].clone(), torch.arange(width, device=DEV)
    fresh = (w >= ((s["before"] + p - 1) // p)[:, None]) & (w < ((s["total"] + p - 1) // p)[:, None])
    free = torch.cat([s["free"], used[fresh].flip(0)])
    used[fresh] = -1
    pages.restore(s["before"], used, free)
    pages.k_cache(0).copy_(s["kc"])
    pages.v_cache(0).copy_(s["vc"])
    if blocks:
        pages.k_scales(0).view(torch.uint8).copy_(s["ks"])
        pages.v_scales(0).view(torch.uint8).copy_(s["vs"])
    elif "sk" in s:
        pages.set_scales(0, s["sk"], s["sv"])
    s["kc"] = s["vc"] = s["ks"] = s["vs"] = None
    pages.plan(s["new"], n + c.get("pad", 0), max_new=s["most_new"])
    return pages


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if op == "norm":
        return _norm_own(s) if own else _norm_plain(s)
    if op == "write":
        return _write_own(s) if own else _write_plain(s)
    return _attention_own(s) if own else _attention_plain(s)


def _norm_own(s):
    from ring_kv_cache_gb300 import residual_norm
    c, mod = s["case"], s["mod"]
    residual_norm(s["h"], s["y"], gate=mod[:, 0] if c["gate"] else None, residual_scale=0.7,
                  post_norm=None if c["post"] == "none" else c["post"], post_weight=s["post_w"], norm=c["kind"],
                  scale=mod[:, 1], shift=mod[:, 2], mod_rows=s["rows"], h_out=s["h_out"], x_out=s["x_out"])
    return [s["h_out"], s["x_out"]]


def _write_own(s):
    c = s["case"]
    qh, kh, d = c["q_heads"], c["kv_heads"], c["dim"]
    q, k, v = s["qkv"].view(-1, qh + 2 * kh, d).split([qh, kh, kh], dim=1)
    pages = s["pages"]
    pages.write(0, q, k, v, q_norm=s["wq"], k_norm=s["wk"], q_out=s["q_out"], pos=s["pos"] if c["axes"] else None)
    out = [s["q_out"], pages.k_cache(0), pages.v_cache(0)]
    return out + [pages.k_scales(0), pages.v_scales(0)] if c["cache"] == "blocks" else out


def _attention_own(s):
    c = s["case"]
    return s["pages"].attention(0, s["q"], out=s["out"], causal=c["causal"], window=c["window"])


def _normed(x, kind, eps=1e-6):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)


def _norm_plain(s):
    c = s["case"]
    mod = s["mod"].float()
    mod = mod[s["rows"].long()] if s["rows"] is not None else mod
    u = s["y"].float()
    if c["post"] != "none":
        u = _normed(u, c["post"]) * s["post_w"].float()
    if c["gate"]:
        u = u * mod[:, 0]
    h = s["h"].float() + 0.7 * u
    s["h_out"].copy_(h)
    s["x_out"].copy_(_normed(h, c["kind"]) * (1.0 + mod[:, 1]) + mod[:, 2])
    return [s["h_out"], s["x_out"]]


def _angles(c, s):
    """cos and sin [t, 1, d / 2] in 32 bits, the angles in 64."""
    d, base = c["dim"], 10000.0
    i = torch.arange(d // 2, device=DEV)
    if not c["axes"]:
        a = s["at"].double()[:, None] * base ** (-2.0 * i.double() / d)
    else:
        tp, yp = c["t_pairs"], c["y_pairs"]
        axis = (i >= tp).long() + (i >= tp + yp).long()
        if c["axes"] == "section":   # each section a rotation of its own
            first, size = _ints([0, tp, tp + yp])[axis], _ints([tp, max(1, yp), d // 2 - tp - yp])[axis]
            theta = base ** (-(i - first).double() / size.double())
        else:
            theta = base ** (-2.0 * i.double() / d)
        a = s["pos"][:c["tokens"]].double()[:, axis] * theta
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate(x, cos, sin, pairing):
    d = x.shape[-1]
    if pairing == "adjacent":
        x0, x1 = x[..., 0::2], x[..., 1::2]
        return torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2)
    x0, x1 = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1)


def _head_norm(x, w):
    return x if w is None else _normed(x, "rms") * w.float()


def _power(amax):
    """The biased exponent of the least power of two s with amax <= 448 s, in [2^-40, 2^40]."""
    m, e = torch.frexp(amax)
    return (torch.where(m <= 0.875, e - 9, e - 8).clamp(-40, 40) + 127).where(amax > 0, 127 - 40)


def _scale(e):
    return torch.exp2(e.float() - 127.0)


def _store_blocks(cache, scales, slots, x):
    """x 32-bit [t, heads, d] at `slots`; blocks that hold tokens before these keep their scale or get a larger one."""
    per = cache.shape[2] // BLOCK
    raw = cache.view(torch.uint8).view(cache.shape[0], cache.shape[1], per, BLOCK, cache.shape[3])
    ids, which = torch.unique(slots // BLOCK, return_inverse=True)
    n, off = len(ids), (slots % BLOCK).long()
    first = torch.full((n,), BLOCK, device=DEV).scatter_reduce(0, which, off, "amin")
    amax = torch.zeros((n, x.shape[1]), device=DEV).scatter_reduce(
        0, which[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    page, sub = (ids // per).long(), (ids % per).long()
    need, old = _power(amax), scales[page, :, sub].to(torch.int32)
    exp = torch.where(first[:, None] > 0, torch.maximum(need, old), need)
    scales[page, :, sub] = exp.to(torch.uint8)
    had = raw[page, :, sub]
    again = _codes(had.view(torch.float8_e4m3fn).float() * torch.exp2((old - exp).float())[:, :, None, None])
    keep = (torch.arange(BLOCK, device=DEV) < first[:, None])[:, None, :, None] & (exp > old)[:, :, None, None]
    raw[page, :, sub] = torch.where(keep, again.view(torch.uint8), had)
    raw[page[which], :, sub[which], off] = _codes(x / _scale(exp)[which][..., None]).view(torch.uint8)


def _store(s, name, x):
    cache, page = s[name + "c"], s["case"]["page"]
    if s["case"]["cache"] == "blocks":
        return _store_blocks(cache, s[name + "s"], s["slots"], x)
    at, off = (s["slots"] // page).long(), (s["slots"] % page).long()
    if s["case"]["cache"] == "bf16":
        cache[at, :, off] = x.to(torch.bfloat16)
    else:
        cache.view(torch.uint8)[at, :, off] = _codes(x * (1.0 / s["s" + name])[:, None]).view(torch.uint8)


def _write_plain(s):
    c = s["case"]
    qh, kh, d, t = c["q_heads"], c["kv_heads"], c["dim"], c["tokens"]
    q, k, v = s["qkv"][:t].float().view(t, qh + 2 * kh, d).split([qh, kh, kh], dim=1)
    cos, sin = _angles(c, s)
    s["q_out"][:t] = _rotate(_head_norm(q, s["wq"]), cos, sin, c["pairing"]).to(torch.bfloat16)
    _store(s, "k", _rotate(_head_norm(k, s["wk"]), cos, sin, c["pairing"]))
    _store(s, "v", v)
    out = [s["q_out"], s["kc"], s["vc"]]
    return out + [s["ks"].view(torch.float8_e8m0fnu), s["vs"].view(torch.float8_e8m0fnu)] if c["cache"] == "blocks" else out


def _attention_plain(s):
    c = s["case"]
    qh, kh, d, p = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    n, total, new, cu = s["q"].shape[0], s["total"].long(), s["new"].long(), s["cu"].long()
    i, j = torch.arange(s["most_new"], device=DEV), torch.arange(s["most_len"], device=DEV)
    q = s["q"][(cu[:-1, None] + i).clamp(max=n - 1)].float().view(len(new), len(i), kh, qh // kh, d)
    page_of, off = s["table"].long()[:, j // p].clamp(min=0), j % p
    there = (j < total[:, None])[:, :, None, None]

    def values(codes, scales):   # [b, j, heads, d] in 32 bits
        x = codes.view(torch.uint8)[page_of, :, off].view(torch.float8_e4m3fn).float()
        return x * _scale(scales[page_of, :, off // BLOCK])[..., None]

    k, v = values(s["kc"], s["ks"]), torch.where(there, values(s["vc"], s["vs"]), 0.0)
    score = torch.einsum("bihgd,bjhd->bhgij", q, k) * d ** -0.5
    pos = (total - new)[:, None] + i
    seen = (j < total[:, None])[:, None, :].expand(-1, len(i), -1)
    if c["causal"]:
        seen = seen & (j <= pos[:, :, None])
        if c["window"]:
            seen = seen & (j > pos[:, :, None] - c["window"])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    score = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    o = torch.einsum("bhgij,bjhd->bihgd", score / score.sum(-1, keepdim=True), v)
    t = torch.arange(n, device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True)
    s["out"].copy_(o[b, t - cu[b]].reshape(n, qh, d).to(torch.bfloat16))
    return s["out"]


# ---------------------------------------------------------------- in 64 bits
def _norm_64(case, s):
    mod = s["mod"].double()
    row = (lambda k: mod[s["rows"].long(), k]) if s["rows"] is not None else (lambda k: mod[0, k])

    def standard(z, kind):
        if kind == "rms":
            return z / torch.sqrt(torch.square(z).sum(1, keepdim=True) / z.shape[1] + 1e-6)
        return (z - z.sum(1, keepdim=True) / z.shape[1]) / torch.sqrt(z.var(1, correction=0, keepdim=True) + 1e-6)

    u = s["y"].double()
    if case["post"] != "none":
        u = standard(u, case["post"]) * s["post_w"].double()
    h = s["h"].double() + 0.7 * (u * row(0) if case["gate"] else u)
    return [h, standard(h, case["kind"]) * (1 + row(1)) + row(2)]


def _write_64(case, s):
    qh, kh, d, p, t = case["q_heads"], case["kv_heads"], case["dim"], case["page"], case["tokens"]
    x = s["qkv"].view(-1, qh + 2 * kh, d).double()
    ang = torch.empty((t, d // 2), dtype=torch.float64, device=DEV)
    ends = [case["t_pairs"], case["t_pairs"] + case["y_pairs"], d // 2]
    for i in range(d // 2):
        if not case["axes"]:
            ang[:, i] = s["at"].double() * math.exp(-math.log(10000.0) * 2 * i / d)
            continue
        ax = next(a for a in range(3) if i < ends[a])
        lo = ends[ax - 1] if ax else 0
        rate = (i - lo) / (ends[ax] - lo) if case["axes"] == "section" else 2 * i / d
        ang[:, i] = s["pos"][:t, ax].double() * math.exp(-math.log(10000.0) * rate)
    turn = torch.polar(torch.ones_like(ang), ang)[:, None]

    def turned(y, w):
        if w is not None:
            y = y / torch.sqrt(torch.square(y).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        if case["pairing"] == "adjacent":
            return torch.view_as_real(torch.view_as_complex(y.reshape(*y.shape[:-1], d // 2, 2)) * turn).flatten(-2)
        z = torch.complex(y[..., :d // 2], y[..., d // 2:]) * turn
        return torch.cat([z.real, z.imag], -1)

    slots = s["slots"].long()
    flat = lambda c: c.to(torch.float64).permute(0, 2, 1, 3).contiguous().view(-1, kh, d)  # noqa: E731  [slot][head][d]
    back = lambda f: f.view(-1, p, kh, d).permute(0, 2, 1, 3).contiguous()  # noqa: E731

    def put(name, y):
        f = flat(s[name + "c"])
        if case["cache"] != "blocks":
            top = 448.0 if case["cache"] == "e4m3" else math.inf
            one = s["s" + name].double() if case["cache"] == "e4m3" else torch.ones(kh, dtype=torch.float64, device=DEV)
            f[slots] = (y / one[:, None]).clamp(-top, top)
            return back(f), None
        # scales as [block][head]; a block's size of the new tokens, its first new place, and what it held
        e = s[name + "s"].permute(0, 2, 1).reshape(-1, kh).double() - 127
        size = torch.zeros((e.shape[0] * BLOCK, kh), dtype=torch.float64, device=DEV)
        size[slots] = y.abs().amax(-1)
        fresh = torch.zeros(e.shape[0] * BLOCK, dtype=torch.bool, device=DEV)
        fresh[slots] = True
        fresh = fresh.view(-1, BLOCK)
        touched = fresh.any(1)
        held = touched & ~fresh[:, 0]
        ends_of = torch.tensor([448.0 * 2.0 ** k for k in range(-40, 40)], dtype=torch.float64, device=DEV)
        want = torch.searchsorted(ends_of, size.view(-1, BLOCK, kh).amax(1)).double() - 40   # the first end not below the size
        after = torch.where(touched[:, None], torch.where(held[:, None], torch.maximum(want, e), want), e)
        before_new = (torch.cumsum(fresh, 1) == 0) & touched[:, None]
        moved = torch.where(before_new[..., None], torch.exp2(e - after)[:, None], 1.0).view(-1, kh)
        f = f * moved[..., None]
        f[slots] = y / torch.exp2(after).repeat_interleave(BLOCK, 0)[slots][..., None]
        return back(f), torch.exp2(after).view(-1, p // BLOCK, kh).permute(0, 2, 1).contiguous()

    q_out = torch.zeros((x.shape[0], qh, d), dtype=torch.float64, device=DEV)
    q_out[:t] = turned(x[:t, :qh], s["wq"])
    (k, ks), (v, vs) = put("k", turned(x[:t, qh:qh + kh], s["wk"])), put("v", x[:t, qh + kh:])
    return [q_out, k, v] + ([ks, vs] if case["cache"] == "blocks" else [])


def _attention_64(case, s):
    qh, kh, d, p = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    before, new = _lengths(case)
    if sum((b + n) * n for b, n in zip(before, new)) * qh * d > 32 * 128 * 4096 * 16384:
        return None
    out, at = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV), 0
    for b, (m, n) in enumerate(zip(before, new)):
        ids = s["table"][b, :-(-(m + n) // p)].long()
        rows = torch.arange(m, m + n, device=DEV)[:, None]
        cols = torch.arange(m + n, device=DEV)[None]
        hide = torch.zeros((n, m + n), dtype=torch.bool, device=DEV)
        if case["causal"]:
            hide = cols > rows
            if case["window"]:
                hide = hide | (rows - cols >= case["window"])
        for h in range(kh):
            k, v = [torch.ldexp(c.view(torch.uint8)[ids, h].view(c.dtype).double().view(-1, BLOCK, d),
                                (e[ids, h].to(torch.int32) - 127).view(-1, 1, 1)).view(-1, d)[:m + n]
                    for c, e in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]
            for g in range(h * (qh // kh), (h + 1) * (qh // kh)):
                w = (s["q"][at:at + n, g].double() @ k.T) / math.sqrt(d)
                out[at:at + n, g] = torch.softmax(w.masked_fill(hide, -math.inf), -1) @ v
        at += n
    return out


def exact(case, seed):
    s = _case(case, seed)
    return {"norm": _norm_64, "write": _write_64, "attention": _attention_64}[case["op"]](case, s)
