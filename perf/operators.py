"""Measured cases of the paged cache: the step's plan (block tables and slot
maps from request lengths), the write (head norms, rotation and quantisation
into the pages) and the attention over the pages.

Each case runs either in its plain form (elementary torch operations in 32
bits, angles in 64) or, with ``own`` set, through ``KvPages``.  Both forms take
what ``prepare`` makes.
"""
import math
import random

import torch

own = False

DEV = "cuda"
HEADS = [(10, 10), (40, 40), (32, 8), (40, 8), (16, 2), (12, 4), (20, 4), (7, 1)]


# ---------------------------------------------------------------- the cases
def listed():
    plan = dict(op="plan")
    write = dict(op="write", norm=True, pad=0)
    att = dict(op="attention", causal=True, window=0)
    return [
        # one new token for each of a small batch: every decode step begins with it
        dict(plan, name="plan_decode", requests=48, long=4000, tokens=48, page=64, lens=1),
        # a large batch in which prompts of up to thousands of tokens join decoding requests
        dict(plan, name="plan_prompts", requests=1000, long=9000, tokens=65536, page=16, lens=2),
        # one decode step of a few requests, the heads of one rank of four
        dict(write, name="write_decode", tokens=9, q_heads=10, kv_heads=10, dim=128, cache="e4m3", pairing="adjacent",
             page=64),
        # one video frame, all heads
        dict(write, name="write_frame", tokens=757, q_heads=40, kv_heads=40, dim=128, cache="e4m3",
             pairing="adjacent", page=64),
        # small heads, an odd number of tokens in a buffer padded for a captured graph, no head norm
        dict(write, name="write_small_heads", tokens=3001, pad=71, q_heads=20, kv_heads=4, dim=64, cache="bf16",
             pairing="halves", page=16, norm=False),
        # a prompt-sized step with shared key/value heads
        dict(write, name="write_prompt", tokens=16384, q_heads=32, kv_heads=8, dim=128, cache="bf16",
             pairing="halves", page=64),
        # a single request that decodes early in its life: latency
        dict(att, name="decode_one", requests=1, new=1, long=700, q_heads=32, kv_heads=8, dim=128, cache="bf16",
             page=64, lens=3),
        # a full batch of decoding requests of ragged lengths
        dict(att, name="decode_batch", requests=128, new=1, long=16384, q_heads=32, kv_heads=8, dim=128, cache="bf16",
             page=64, lens=4),
        # few long requests in eight bits, no shared heads, a few tokens each (drafts being checked)
        dict(att, name="decode_drafts", requests=6, new=4, long=32000, q_heads=10, kv_heads=10, dim=128, cache="e4m3",
             page=16, lens=5),
        # one frame over the filled window, every token sees every other
        dict(att, name="frame", requests=1, new=757, long=5788, q_heads=40, kv_heads=40, dim=128, cache="e4m3",
             page=64, lens=6, causal=False),
        # a chunk of a long prompt behind what is cached
        dict(att, name="chunk", requests=1, new=4096, long=16384, q_heads=32, kv_heads=8, dim=128, cache="bf16",
             page=64, lens=7),
        # ragged chunks of several requests, a sliding window, small heads
        dict(att, name="chunks_window", requests=11, new=900, long=5000, q_heads=20, kv_heads=4, dim=64, cache="bf16",
             page=32, lens=8, window=1500),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng, dim):
    return rng.choice([h for h in HEADS if (h[0] + 2 * h[1]) * dim <= 120 * 128])


def draw(rng):
    kind = rng.choice(["plan", "write", "attention", "attention"])
    if kind == "plan":
        b = _log(rng, 1, 1000)
        return dict(op="plan", requests=b, long=_log(rng, 64, 9000), tokens=max(b, _log(rng, 1, 65536)),
                    page=rng.choice([16, 32, 64, 128, 256]), lens=rng.randrange(10 ** 6))
    dim = rng.choice([64, 128, 128])
    qh, kh = _heads(rng, dim)
    c = dict(op=kind, q_heads=qh, kv_heads=kh, dim=dim, cache=rng.choice(["e4m3", "bf16"]),
             page=rng.choice([16, 32, 64, 128, 256]))
    if kind == "write":
        most = 16384 * 48 * 128 // ((qh + 2 * kh) * dim)
        t = _log(rng, 1, min(16384, most))
        return dict(c, tokens=t, pad=rng.choice([0, 0, 13]), norm=rng.random() < 0.75,
                    pairing=rng.choice(["adjacent", "halves"]))
    c["lens"] = rng.randrange(10 ** 6)
    if rng.random() < 0.5:   # single tokens and drafts
        new = rng.choice([1, 1, 1, 2, 3, 5])
        long = _log(rng, max(8, new), 32000)
        most = max(1, min(128, 128 * 16384 * 8 * 128 // (long * kh * dim), 2 ** 31 // (long * qh * new)))
        return dict(c, requests=_log(rng, 1, most), new=new, long=long, causal=True,
                    window=rng.choice([0, 0, 0, 500]))
    new = _log(rng, 6, 4096)
    long = _log(rng, new, 16384)
    full = 26 * 4096 * 16384   # query rows x keys
    long = max(new, min(long, full // (qh * new)))
    most = max(1, min(16, full // (long * qh * new)))
    return dict(c, requests=_log(rng, 1, most), new=new, long=long, causal=rng.random() < 0.75,
                window=0)


def _lengths(case):
    """(cached before the step, new) of every request, from the case alone."""
    r = random.Random(case["lens"])
    n = case["requests"]
    if case["op"] == "plan":
        long, tokens = case["long"], case["tokens"]
        new = [1] * n
        left = tokens - n
        while left > 0:   # prompts of various lengths until the step is full, or nearly
            i, x = r.randrange(n), min(left, _log(r, 1, max(1, long)))
            new[i] += x
            left -= max(x, 1 + tokens // 4096)
        return [r.randrange(0, long + 1) for _ in range(n)], new
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
    full = before + new
    grow = max(0, min(new, w - before))       # tokens whose window still reaches back to the start
    return grow * before + grow * (grow + 1) // 2 + (new - grow) * w, min(full, new - 1 + w)


def work(case):
    if case["op"] == "plan":
        before, new = _lengths(case)
        p = case["page"]
        pages = sum(-(-(b + n) // p) - -(-b // p) for b, n in zip(before, new))
        return {"bytes": 12 * len(new) + 4 * pages + 8 * len(new) + 4 * pages + 8 * case["tokens"], "flops": 0}
    qh, kh, d = case["q_heads"], case["kv_heads"], case["dim"]
    size = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "write":
        t = case["tokens"]
        return {"bytes": t * d * (2 * (qh + 2 * kh) + 2 * qh + size * 2 * kh) + 8 * t + 4 * d * t,
                "flops": 8 * t * d * (qh + kh)}
    before, new = _lengths(case)
    both = [_pairs(case, b, n) for b, n in zip(before, new)]
    return {"bytes": 4 * d * qh * sum(new) + 2 * size * d * kh * sum(k for _, k in both),
            "flops": 4 * d * qh * sum(p for p, _ in both)}


# ---------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _codes(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _tables(total, extra, page, g, spare):
    """Block tables of requests of the given lengths in a shuffled pool, and the pages left over."""
    need = [-(-t // page) for t in total]
    width = max(1, max(-(-(t + e) // page) for t, e in zip(total, extra)))
    num = sum(need) + spare
    order = torch.randperm(num, generator=g, device=DEV).to(torch.int32)
    n = torch.tensor(need, device=DEV)
    first = torch.cumsum(n, 0) - n
    w = torch.arange(width, device=DEV)
    at = (first[:, None] + w).clamp(max=num - 1)
    table = torch.where(w < n[:, None], order[at], torch.full((), -1, dtype=torch.int32, device=DEV))
    return table.contiguous(), order[sum(need):].contiguous(), num


def _pool(case, num, g):
    shape = (num, case["kv_heads"], case["page"], case["dim"])
    big = case["cache"] == "e4m3"

    def one():
        x = torch.empty(shape, dtype=torch.float8_e4m3fn if big else torch.bfloat16, device=DEV)
        for i in range(0, num, 4096):   # no 32-bit copy of a whole large pool
            y = torch.randn((min(4096, num - i),) + shape[1:], generator=g, device=DEV)
            x[i:i + 4096] = _codes(y * 100.0) if big else y.to(torch.bfloat16)
        return x

    return one(), one()


def _scales(case, g):
    if case["cache"] != "e4m3":
        return None, None
    one = lambda: 0.005 + 0.01 * torch.rand(case["kv_heads"], generator=g, device=DEV)  # noqa: E731
    return one(), one()


def _case(case, seed):
    """The tensors of a case, the same for every form."""
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "plan":
        before, new = _lengths(case)
        order = list(range(len(new)))
        random.Random(seed).shuffle(order)   # which request holds which row of the tables
        p = case["page"]
        taken = sum(-(-(b + n) // p) - -(-b // p) for b, n in zip(before, new))
        back = [0] * len(new)
        for b, row in enumerate(order):
            back[row] = b
        table, free, num = _tables([before[b] for b in back], [new[b] for b in back], p, g, taken + 37)
        s.update(table=table, free=free, num=num, lens=torch.tensor([before[b] for b in back], dtype=torch.int32, device=DEV),
                 rows=torch.tensor(order, dtype=torch.int32, device=DEV), new=torch.tensor(new, dtype=torch.int32, device=DEV))
        return s
    qh, kh, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "write":
        t, pad, p = case["tokens"], case["pad"], case["page"]
        cols = (qh + 2 * kh) * d
        qkv = torch.randn((t + pad, cols), generator=g, device=DEV).to(torch.bfloat16)
        qkv = qkv * (0.5 + 2.0 * torch.rand((1, cols), generator=g, device=DEV)).to(torch.bfloat16)
        before = 1217
        table, free, num = _tables([before + t], [0], p, g, 3)
        kc, vc = _pool(case, num, g)
        s.update(qkv=qkv, table=table, free=free, num=num, kc=kc, vc=vc, before=before,
                 q_out=torch.zeros((t + pad, qh, d), dtype=torch.bfloat16, device=DEV))
        s["sk"], s["sv"] = _scales(case, g)
        s["wq"], s["wk"] = [(0.5 + torch.rand(d, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None
                            for _ in range(2)]
        pos = torch.arange(before, before + t, device=DEV)
        slots = table[0, pos // p] * p + (pos % p).to(torch.int32)
        s.update(pos=pos.to(torch.int32), slots=slots)
        return s
    before, new = _lengths(case)
    total = [b + n for b, n in zip(before, new)]
    table, free, num = _tables(total, [0] * len(new), case["page"], g, 5)
    kc, vc = _pool(case, num, g)
    q = (1.5 * torch.randn((sum(new), qh, d), generator=g, device=DEV)).to(torch.bfloat16)
    s.update(q=q, table=table, free=free, num=num, kc=kc, vc=vc, most_new=max(new), most_len=max(total),
             before=torch.tensor(before, dtype=torch.int32, device=DEV),
             total=torch.tensor(total, dtype=torch.int32, device=DEV), new=torch.tensor(new, dtype=torch.int32, device=DEV),
             cu=torch.cumsum(torch.tensor([0] + new, device=DEV), 0).to(torch.int32),
             out=torch.zeros_like(q))
    s["sk"], s["sv"] = _scales(case, g)
    return s


def prepare(case, seed):
    s = _case(case, seed)
    if own:
        s["pages"] = _pages(s)
    return s


def _pages(s):
    """The cache a program keeps, in the state that the case's tensors describe."""
    from ring_kv_cache_gb300 import KvPages
    c = s["case"]
    rows, width = s["table"].shape
    dt = torch.float8_e4m3fn if c.get("cache") == "e4m3" else torch.bfloat16
    pages = KvPages(c.get("q_heads", 1), c.get("kv_heads", 1), c.get("dim", 64), page_size=c["page"],
                    num_pages=s["num"], max_requests=rows, max_request_tokens=width * c["page"],
                    max_tokens=c.get("tokens", 0) + c.get("pad", 0) or s["q"].shape[0], cache_dtype=dt,
                    rope_pairing=c.get("pairing", "adjacent"))
    used = s["table"][:, :].clone()
    if c["op"] == "plan":
        lens = s["lens"]
    elif c["op"] == "write":
        lens = torch.full((1,), s["before"], dtype=torch.int32, device=DEV)
    else:
        lens = s["before"]
    if c["op"] != "plan":
        # the step's own new pages are the next ones the plan takes: back onto the free list in its order
        p = c["page"]
        end = s["total"] if c["op"] == "attention" else lens + c["tokens"]
        w = torch.arange(width, device=DEV)
        fresh = (w >= ((lens + p - 1) // p)[:, None]) & (w < ((end + p - 1) // p)[:, None])
        free = torch.cat([s["free"], used[fresh].flip(0)])
        used[fresh] = -1
    else:
        free = s["free"]
    pages.restore(lens, used, free)
    if "kc" in s:
        pages.k_cache(0).copy_(s["kc"])
        pages.v_cache(0).copy_(s["vc"])
        s["kc"] = s["vc"] = None
        if s["sk"] is not None:
            pages.set_scales(0, s["sk"], s["sv"])
    if c["op"] == "write":
        pages.plan(torch.full((1,), c["tokens"], dtype=torch.int32, device=DEV), c["tokens"] + c["pad"])
    elif c["op"] == "attention":
        pages.plan(s["new"], s["q"].shape[0], max_new=s["most_new"])
    return pages


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if c["op"] == "plan":
        return _plan_own(s) if own else _plan_plain(s)
    if c["op"] == "write":
        return _write_own(s) if own else _write_plain(s)
    return _attention_own(s) if own else _attention_plain(s)


def _plan_own(s):
    step = s["pages"].plan(s["new"], s["case"]["tokens"], rows=s["rows"])
    return [step.cu, step.lengths, step.positions, step.slots, s["pages"].tables]


def _write_own(s):
    c = s["case"]
    qh, kh, d = c["q_heads"], c["kv_heads"], c["dim"]
    q, k, v = s["qkv"].view(-1, qh + 2 * kh, d).split([qh, kh, kh], dim=1)
    s["pages"].write(0, q, k, v, q_norm=s["wq"], k_norm=s["wk"], q_out=s["q_out"])
    return [s["q_out"], s["pages"].k_cache(0), s["pages"].v_cache(0)]


def _attention_own(s):
    c = s["case"]
    return s["pages"].attention(0, s["q"], out=s["out"], causal=c["causal"], window=c["window"])


def _plan_plain(s):
    p, t = s["case"]["page"], s["case"]["tokens"]
    rows, new, free, table = s["rows"].long(), s["new"].long(), s["free"], s["table"]
    lens = s["lens"].long()[rows]
    after = lens + new
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(new, 0)])
    have, need = (lens + p - 1) // p, (after + p - 1) // p
    n = need - have
    off = torch.cumsum(n, 0) - n
    w = torch.arange(table.shape[1], device=DEV)
    at = free.numel() - 1 - (off[:, None] + w - have[:, None])
    fresh = (w >= have[:, None]) & (w < need[:, None])
    table[rows] = torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table[rows])
    i = torch.arange(t, device=DEV)
    b = torch.searchsorted(cu[1:], i, right=True).clamp(max=len(new) - 1)
    inside = i < cu[-1]
    pos = torch.where(inside, lens[b] + i - cu[b], 0)
    slot = torch.where(inside, table[rows[b], pos // p] * p + pos % p, -1)
    return [cu.int(), after.int(), pos.int(), slot.int(), table]


def _rotate(x, pos, pairing, base=10000.0):
    """x: 32-bit [t, heads, d]; the angles in 64 bits."""
    d = x.shape[-1]
    theta = base ** (-torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)
    a = pos.double()[:, None] * theta
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    if pairing == "adjacent":
        x0, x1 = x[..., 0::2], x[..., 1::2]
        return torch.stack([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1).flatten(-2)
    x0, x1 = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([x0 * cos - x1 * sin, x0 * sin + x1 * cos], -1)


def _norm(x, w, eps=1e-6):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _store(cache, slots, x, scale):
    page = cache.shape[2]
    at, off = (slots // page).long(), (slots % page).long()
    if scale is None:
        cache[at, :, off] = x.to(torch.bfloat16)
    else:
        cache.view(torch.uint8)[at, :, off] = _codes(x * (1.0 / scale)[:, None]).view(torch.uint8)


def _write_plain(s):
    c = s["case"]
    qh, kh, d, t = c["q_heads"], c["kv_heads"], c["dim"], c["tokens"]
    q, k, v = s["qkv"][:t].float().view(t, qh + 2 * kh, d).split([qh, kh, kh], dim=1)
    s["q_out"][:t] = _rotate(_norm(q, s["wq"]), s["pos"], c["pairing"]).to(torch.bfloat16)
    _store(s["kc"], s["slots"], _rotate(_norm(k, s["wk"]), s["pos"], c["pairing"]), s["sk"])
    _store(s["vc"], s["slots"], v, s["sv"])
    return [s["q_out"], s["kc"], s["vc"]]


def _gather(cache, page_of, off):
    """Cached rows [b, j, heads, d] in 32 bits."""
    if cache.dtype == torch.bfloat16:
        return cache[page_of, :, off].float()
    return cache.view(torch.uint8)[page_of, :, off].view(torch.float8_e4m3fn).float()


def _attention_plain(s):
    c = s["case"]
    qh, kh, d, p = c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    n, total, new, cu = s["q"].shape[0], s["total"].long(), s["new"].long(), s["cu"].long()
    i, j = torch.arange(s["most_new"], device=DEV), torch.arange(s["most_len"], device=DEV)
    q = s["q"][(cu[:-1, None] + i).clamp(max=n - 1)].float().view(len(new), len(i), kh, qh // kh, d)
    page_of, off = s["table"].long()[:, j // p].clamp(min=0), j % p
    there = (j < total[:, None])[:, :, None, None]
    k, v = _gather(s["kc"], page_of, off), torch.where(there, _gather(s["vc"], page_of, off), 0.0)
    if s["sk"] is not None:
        k, v = k * s["sk"][:, None], v * s["sv"][:, None]
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
def exact(case, seed):
    if case["op"] == "plan":   # whole numbers alone
        return None
    s = _case(case, seed)
    qh, kh, d, p = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    one = [torch.ones(kh, device=DEV)] * 2
    sk, sv = [(a if a is not None else b).double() for a, b in zip((s["sk"], s["sv"]), one)]
    if case["op"] == "write":
        t = case["tokens"]
        x = s["qkv"].view(-1, qh + 2 * kh, d).double()
        freq = torch.exp(-math.log(10000.0) * 2 * torch.arange(d // 2, device=DEV, dtype=torch.float64) / d)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["pos"].double()[:, None, None] * freq)

        def turned(y, w):
            if w is not None:
                y = y / torch.sqrt(torch.square(y).sum(-1, keepdim=True) / d + 1e-6) * w.double()
            if case["pairing"] == "adjacent":
                return torch.view_as_real(torch.view_as_complex(y.reshape(*y.shape[:-1], d // 2, 2)) * turn).flatten(-2)
            z = torch.complex(y[..., :d // 2], y[..., d // 2:]) * turn
            return torch.cat([z.real, z.imag], -1)

        def put(cache, y, scale):
            full = cache.to(torch.float64)
            top = 448.0 if case["cache"] == "e4m3" else math.inf
            flat = full.permute(0, 2, 1, 3).contiguous().view(-1, kh, d)   # [slot][head][d]
            flat[s["slots"].long()] = (y / scale[:, None]).clamp(-top, top)
            return flat.view(-1, p, kh, d).permute(0, 2, 1, 3).contiguous()

        q_out = torch.zeros((x.shape[0], qh, d), dtype=torch.float64, device=DEV)
        q_out[:t] = turned(x[:t, :qh], s["wq"])
        return [q_out, put(s["kc"], turned(x[:t, qh:qh + kh], s["wk"]), sk), put(s["vc"], x[:t, qh + kh:], sv)]
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
            if s["kc"].dtype == torch.bfloat16:
                k, v = s["kc"][ids, h], s["vc"][ids, h]
            else:
                k, v = [x.view(torch.uint8)[ids, h].view(x.dtype) for x in (s["kc"], s["vc"])]
            k = k.double().reshape(-1, d)[:m + n] * sk[h]
            v = v.double().reshape(-1, d)[:m + n] * sv[h]
            for g in range(h * (qh // kh), (h + 1) * (qh // kh)):
                w = (s["q"][at:at + n, g].double() @ k.T) / math.sqrt(d)
                out[at:at + n, g] = torch.softmax(w.masked_fill(hide, -math.inf), -1) @ v
        at += n
    return out
