"""Plain 64-bit forms of the paged cache's operators and the error each kernel
may make, for the GPU tests.

Roundings are off by at most half a step: bf16 2^-8, f16 2^-11, E4M3 2^-4
relative (E4M3 below 2^-6: 2^-10 absolute).
"""
import math

import numpy as np
import torch

import ring_kv_cache_gb300 as kv

F64 = torch.float64


class Allocator:
    """The block tables on the host, one page at a time."""

    def __init__(self, rows, width, page, num_pages):
        self.page, self.width = page, width
        self.lens = [0] * rows
        self.table = [[-1] * width for _ in range(rows)]
        self.free = list(range(num_pages - 1, -1, -1))

    def plan(self, rows, new, num_tokens):
        """(cu, lengths, positions, slots, {(row, w): page}, taken) or None if it cannot be made."""
        free = list(self.free)
        cu, lens, pos, slots, fresh = [0], [], [], [], {}
        if len(set(rows)) != len(rows) or sum(new) > num_tokens or min(new) < 0:
            return None
        for r, n in zip(rows, new):
            if self.lens[r] + n > self.width * self.page:
                return None
            for w in range(-(-self.lens[r] // self.page), -(-(self.lens[r] + n) // self.page)):
                if not free:
                    return None
                fresh[r, w] = free.pop()
            for p in range(self.lens[r], self.lens[r] + n):
                w = p // self.page
                pos.append(p)
                slots.append(fresh.get((r, w), self.table[r][w]) * self.page + p % self.page)
            cu.append(cu[-1] + n)
            lens.append(self.lens[r] + n)
        pad = num_tokens - len(pos)
        return cu, lens, pos + [0] * pad, slots + [-1] * pad, fresh, len(self.free) - len(free)

    def commit(self, rows, plan):
        _, lens, _, _, fresh, taken = plan
        for r, n in zip(rows, lens):
            self.lens[r] = n
        for (r, w), p in fresh.items():
            self.table[r][w] = p
        if taken:
            del self.free[-taken:]

    def release(self, rows):
        for r in rows:
            for w in range(-(-self.lens[r] // self.page)):
                self.free.append(self.table[r][w])
                self.table[r][w] = -1
            self.lens[r] = 0


def filled(hq, hkv, d, page, total, new, cache, seed=0, layers=1, layer=0, spare=3, pairing="adjacent", garbage=True,
           pad=0, magnitude=1.0):
    """A cache in which request i holds total[i] tokens, the last new[i] of
    them planned as the step's; pages shuffled, places no token has reached
    full of NaN.  Returns (pages, state dict)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    need = [-(-t // page) for t in total]
    num = sum(need) + spare
    width = max(1, max(need))
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32).cpu().tolist()
    table = [[-1] * width for _ in total]
    at, back = 0, []
    before = [t - n for t, n in zip(total, new)]
    for b, t in enumerate(total):
        for w in range(need[b]):
            if w * page < -(-before[b] // page) * page:
                table[b][w] = order[at]
            else:
                back.append(order[at])
            at += 1
    free = order[at:] + back[::-1]
    dt = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    tokens = max(1, sum(new)) + pad
    p = kv.KvPages(hq, hkv, d, page_size=page, num_pages=num, max_requests=len(total), max_request_tokens=width * page,
                   max_tokens=tokens, layers=layers, cache_dtype=dt, rope_pairing=pairing)
    i32 = dict(dtype=torch.int32, device="cuda")
    p.restore(torch.tensor(before, **i32), torch.tensor(table, **i32),
              torch.tensor(free, **i32) if free else torch.zeros(0, **i32))
    s = dict(total=total, new=new, before=before, layer=layer)
    if cache == "e4m3":
        s["sk"] = (0.005 + 0.01 * torch.rand(hkv, generator=g, device="cuda")) * magnitude
        s["sv"] = 0.005 + 0.01 * torch.rand(hkv, generator=g, device="cuda")
        p.set_scales(layer, s["sk"], s["sv"])
    p.plan(torch.tensor(new, **i32), tokens, max_new=max(1, max(new)))
    for c, m in ((p.k_cache(layer), 1.0 if cache == "e4m3" else magnitude), (p.v_cache(layer), 1.0)):
        x = torch.randn(c.shape, generator=g, device="cuda") * (100.0 if cache == "e4m3" else m)
        if garbage:   # what no token has reached
            used = torch.zeros((num, page), dtype=torch.bool, device="cuda")
            tab = p.tables.tolist()
            for b, t in enumerate(total):
                for w in range(need[b]):
                    used[tab[b][w], :min(page, t - w * page)] = True
            x = torch.where(used[:, None, :, None], x, math.nan)
        c.copy_(x.clamp(-448, 448).to(dt) if cache == "e4m3" else x.to(dt))
    s["q"] = (1.5 * torch.randn((tokens, hq, d), generator=g, device="cuda")).to(torch.bfloat16)
    return p, s


def cached(p, s, b, h, which):
    """float64 [total, d]: request b's cached keys or values of head h."""
    c = (p.k_cache if which == "k" else p.v_cache)(s["layer"])
    n = s["total"][b]
    ids = p.tables[b, :-(-n // p.P)].long()
    raw = c.view(torch.uint8) if c.dtype == torch.float8_e4m3fn else c
    x = raw[ids, h]
    x = (x.view(c.dtype) if c.dtype == torch.float8_e4m3fn else x).to(F64).reshape(-1, p.d)[:n]
    return x * s["s" + which][h].double() if "s" + which in s else x


def attention_64(p, s, q=None, causal=True, window=0, scale=None):
    """(out, bound) in 64 bits, NaN in rows past the plan's tokens."""
    q = s["q"] if q is None else q
    sm = scale or 1 / math.sqrt(p.d)
    e4m3 = p.cache_dtype == torch.float8_e4m3fn
    G = p.Hq // p.Hkv
    out = torch.full(q.shape, math.nan, dtype=F64, device="cuda")
    tol = torch.zeros_like(out)
    at = 0
    for b, (t, n) in enumerate(zip(s["total"], s["new"])):
        if n == 0:
            continue
        i, j = torch.arange(t - n, t, device="cuda")[:, None], torch.arange(t, device="cuda")[None]
        see = torch.ones((n, t), dtype=torch.bool, device="cuda")
        if causal:
            see = (j <= i) & ((j > i - window) if window else True)
        for h in range(p.Hq):
            k, v = cached(p, s, b, h // G, "k"), cached(p, s, b, h // G, "v")
            x = q[at:at + n, h].double()
            w = torch.softmax((x @ k.T * sm).masked_fill(~see, -math.inf), -1)
            vv = torch.where(see.any(0)[:, None], v, 0.0)
            o = w @ vv
            a = w @ vv.abs()
            # a score's fp32 sum over d products (2^-22 each with the tensor
            # cores' truncation) and, over E4M3, the query's f16 form (2^-25
            # of its row's largest)
            size = (x.abs() @ k.abs().T).masked_fill(~see, 0).amax(-1, keepdim=True) * sm
            delta = size * p.d * 2.0 ** -22 + 2.0 ** -20
            if e4m3:
                delta = delta + 2.0 ** -24 * x.abs().amax(-1, keepdim=True) * k.abs().sum(-1).amax() * sm
            # probabilities to 16 bits (f16: 2^-25 absolute below 2^-14, of a
            # largest one of 1), the result to bf16, the fp32 sums over tokens
            lost = (2.0 ** -11 if e4m3 else 2.0 ** -8) + 2 * delta + 2.0 ** -22 * math.sqrt(t)
            tol[at:at + n, h] = 2.0 ** -8 * o.abs() + lost * a * 1.01 + 1e-30
            if e4m3:
                tol[at:at + n, h] += t * 2.0 ** -25 * vv.abs().max()
            out[at:at + n, h] = o
        at += n
    return out, tol


def norm_rope_64(x, w, pos, pairing, eps=1e-6, base=10000.0):
    """float64 [n, heads, d] normed and rotated, and the sizes |a| + |b| of what each value is made of."""
    y = x.double()
    d = y.shape[-1]
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    if pos is None:
        return y, y.abs()
    theta = torch.tensor([base ** (-2 * i / d) for i in range(d // 2)], dtype=F64, device=x.device)
    ang = pos.double()[:, None, None] * theta
    c, s = ang.cos(), ang.sin()
    a, b = (y[..., 0::2], y[..., 1::2]) if pairing == "adjacent" else (y[..., :d // 2], y[..., d // 2:])
    r0, r1, m = a * c - b * s, a * s + b * c, a.abs() + b.abs()
    if pairing == "adjacent":
        return torch.stack([r0, r1], -1).flatten(-2), torch.stack([m, m], -1).flatten(-2)
    return torch.cat([r0, r1], -1), torch.cat([m, m], -1)


def close(got, want, tol, what=""):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(((got.double() - want).abs() / tol).nan_to_num(9e9).max()),
                           bad.nonzero()[:3].tolist())


def errors(p):
    return int(p.state[kv.PAGES_STATE["error"]].item())


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")
