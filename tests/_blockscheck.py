"""Caches with block scales or 3-D positions for the GPU tests, and their plain
64-bit forms.  A block is 16 tokens of a page; its scale is 2^(byte - 127)."""
import math

import torch

import ring_kv_cache_gb300 as kv
from _pagescheck import F64

B = kv.SCALE_BLOCK
LOW, HIGH = 127 - 40, 127 + 40


def cache_of(hq, hkv, d, page, total, new, seed=0, layers=1, layer=0, spare=3, pairing="adjacent", pad=0,
             cache="blocks", low=-9, high=-4, rope3d=None, frequencies="section", max_position=None, missing=(), garbage=True):
    """A cache in which request i holds total[i] tokens, the last new[i] of
    them planned as the step's; pages shuffled, pages `missing` (request, place)
    not of the pool; places no token has reached full of NaN codes.  Returns
    (pages, state)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-t // page) for t in total]
    num = max(1, sum(need) + spare)
    width = max(1, max(need))
    order = torch.randperm(num, generator=g, device="cuda").tolist()
    table, back, at = [[-1] * width for _ in total], [], 0
    before = [t - n for t, n in zip(total, new)]
    for b in range(len(total)):
        for w in range(need[b]):
            if w * page < -(-before[b] // page) * page:
                table[b][w] = order[at] if (b, w) not in missing else num + 7
            else:
                back.append(order[at] if (b, w) not in missing else -3)
            at += 1
    free = order[at:] + back[::-1]
    tokens = max(1, sum(new)) + pad
    three = dict(rope3d=rope3d, rope_frequencies=frequencies, max_position=max_position) if rope3d else {}
    p = kv.KvPages(hq, hkv, d, page_size=page, num_pages=num, max_requests=len(total), max_request_tokens=width * page,
                   max_tokens=tokens, layers=layers, cache_dtype=torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn,
                   rope_pairing=pairing, block_scales=cache == "blocks", **three)
    i32 = dict(dtype=torch.int32, device="cuda")
    p.restore(torch.tensor(before, **i32), torch.tensor(table, **i32),
              torch.tensor(free, **i32) if free else torch.zeros(0, **i32))
    s = dict(total=total, new=new, before=before, layer=layer, tokens=sum(new))
    if cache == "e4m3":
        s["sk"], s["sv"] = [0.005 + 0.01 * torch.rand(hkv, generator=g, device="cuda") for _ in range(2)]
        p.set_scales(layer, s["sk"], s["sv"])
    p.plan(torch.tensor(new, **i32), tokens, max_new=max(1, max(new)))
    used = torch.zeros((num, page), dtype=torch.bool, device="cuda")
    for b, t in enumerate(total):
        for w in range(need[b]):
            if (b, w) not in missing:
                used[p.tables[b, w], :min(page, t - w * page)] = True
    for c in (p.k_cache(layer), p.v_cache(layer)):
        x = torch.randn(c.shape, generator=g, device="cuda") * (1.0 if cache == "bf16" else 100.0)
        if garbage:
            x = torch.where(used[:, None, :, None], x, math.nan)
        c.copy_(x.clamp(-448, 448).to(c.dtype) if cache != "bf16" else x.to(c.dtype))
    if cache == "blocks":
        for sc in (p.k_scales(layer), p.v_scales(layer)):
            e = 127 + torch.randint(low, high, sc.shape, generator=g, device="cuda")
            if garbage:   # blocks no token has reached
                e = torch.where(used.view(num, 1, page // B, B).any(-1), e, torch.randint(0, 256, sc.shape, generator=g, device="cuda"))
            sc.view(torch.uint8).copy_(e.to(torch.uint8))
    s["q"] = (1.5 * torch.randn((tokens, hq, d), generator=g, device="cuda")).to(torch.bfloat16)
    return p, s


def turned(x, w, angles, pairing, eps=1e-6):
    """float64 [n, heads, d] normed (weights w or None) and turned by angles
    [n, d/2] (None: not), and the sizes of what each value is made of."""
    y = x.double()
    d = y.shape[-1]
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    if angles is None:
        return y, y.abs()
    c, s = angles.cos()[:, None], angles.sin()[:, None]
    a, b = (y[..., 0::2], y[..., 1::2]) if pairing == "adjacent" else (y[..., :d // 2], y[..., d // 2:])
    r = [a * c - b * s, a * s + b * c]
    m = [a.abs() + b.abs()] * 2
    join = (lambda z: torch.stack(z, -1).flatten(-2)) if pairing == "adjacent" else (lambda z: torch.cat(z, -1))
    return join(r), join(m)


def angles_of(d, pos, rope3d=None, frequencies="section", base=10000.0):
    """float64 [n, d/2]: pos [n], or [n, 3] with rope3d."""
    if rope3d is None:
        return pos.double()[:, None] * torch.tensor([base ** (-2 * i / d) for i in range(d // 2)], dtype=F64, device=pos.device)
    ends = [0, rope3d[0], rope3d[0] + rope3d[1], d // 2]
    cols = []
    for i in range(d // 2):
        a = max(k for k in range(3) if ends[k] <= i and ends[k + 1] > i)
        rate = (i - ends[a]) / (ends[a + 1] - ends[a]) if frequencies == "section" else 2 * i / d
        cols.append(pos[:, a].double() * base ** -rate)
    return torch.stack(cols, 1)


def exponents(amax):
    """Biased least exponents e with amax <= 448 * 2^(e - 127), as documented."""
    ends = torch.tensor([448.0 * 2.0 ** k for k in range(-40, 40)], dtype=F64, device=amax.device)
    return torch.searchsorted(ends, amax.double().contiguous()) + LOW


def check_blocks(p, s, name, want, m, slots, planned, before, scales_before, fp=2.0 ** -19):
    """The cache after a write of `want` (float64 [n, heads, d], sizes m) at `slots`
    (-1: a token that was skipped), of those `planned`."""
    layer = s["layer"]
    cache = (p.k_cache if name == "k" else p.v_cache)(layer)
    sc = (p.k_scales if name == "k" else p.v_scales)(layer).view(torch.uint8)
    per, d, H = p.P // B, p.d, p.Hkv
    view = lambda c: c.view(torch.uint8).view(p.num_pages, H, per, B, d).transpose(1, 2).reshape(-1, H, B, d)  # noqa: E731
    got, old = view(cache), view(before)
    e_got = sc.transpose(1, 2).reshape(-1, H).long()
    e_old = scales_before.transpose(1, 2).reshape(-1, H).long()
    dec = lambda u: u.contiguous().view(torch.float8_e4m3fn).double()  # noqa: E731
    written, begin = {}, {}
    for i, (sl, pl) in enumerate(zip(slots.tolist(), planned.tolist())):
        if pl >= 0:
            begin.setdefault(pl // B, pl % B)   # the block's places before this one held tokens
        if sl >= 0:
            written.setdefault(sl // B, []).append((sl % B, i))
    touched = torch.zeros(got.shape[0], dtype=torch.bool, device="cuda")
    for blk, rows in written.items():
        touched[blk] = True
        off, idx = [r[0] for r in rows], [r[1] for r in rows]
        first = begin[blk]
        x, size = want[idx], m[idx]                          # [n, H, d]
        fin = torch.where(torch.isfinite(x), x.abs(), 0.0)
        amax = fin.amax((0, 2))
        err = fp * size.amax((0, 2)) if name == "k" else torch.zeros_like(amax)
        lo, hi = exponents((amax - err).clamp(min=0)), exponents(amax + err)
        if first > 0:
            so_far = e_old[blk].clamp(LOW, HIGH)
            lo, hi = torch.maximum(lo, so_far), torch.maximum(hi, so_far)
        e = e_got[blk]
        assert bool(((e >= lo) & (e <= hi)).all()), (name, blk, e.tolist(), lo.tolist(), hi.tolist())
        scale = torch.exp2(e.double() - 127)
        val = dec(got[blk][:, off]) * scale[:, None, None]    # [H, n, d]
        x, size = x.transpose(0, 1), size.transpose(0, 1)
        top = (448 * scale)[:, None, None]
        clipped = torch.minimum(torch.maximum(x, -top), top)
        tol = 2.0 ** -4 * clipped.abs() + 2.0 ** -10 * scale[:, None, None] + (fp * size if name == "k" else 0)
        ok = ((val - clipped).abs() <= tol) | (torch.isnan(x) & torch.isnan(val))
        assert bool(ok.all()), (name, blk, (~ok).nonzero()[:3].tolist())
        if first > 0:                                         # what the block held before
            had = old[blk][:, :first]
            ratio = torch.exp2((e_old[blk].clamp(LOW, HIGH) - e).float())[:, None, None]
            again = (dec(had).float() * ratio).to(torch.float8_e4m3fn).view(torch.uint8)
            moved = (e > e_old[blk].clamp(LOW, HIGH))[:, None, None]
            assert torch.equal(got[blk][:, :first], torch.where(moved, again, had)), (name, blk)
        rest = [k for k in range(first, B) if k not in off]   # places of nobody
        assert torch.equal(got[blk][:, rest], old[blk][:, rest])
    assert torch.equal(got[~touched], old[~touched]) and torch.equal(e_got[~touched], e_old[~touched])


def cached_blocks(p, s, b, h, which):
    """float64 (codes [total, d], scales [total]) of request b's head h."""
    layer, n = s["layer"], s["total"][b]
    c, sc = [getattr(p, which + x)(layer).view(torch.uint8) for x in ("_cache", "_scales")]
    ids = p.tables[b, :-(-n // p.P)].long()
    codes = c[ids, h].view(torch.float8_e4m3fn).double().reshape(-1, p.d)[:n]
    e = sc[ids, h].long().clamp(LOW, HIGH).repeat_interleave(B, dim=1).reshape(-1)[:n]
    return codes, torch.exp2(e.double() - 127)


def attention_blocks_64(p, s, q=None, causal=True, window=0, scale=None):
    """(out, bound) in 64 bits, NaN in rows past the plan's tokens."""
    q = s["q"] if q is None else q
    sm = scale or 1 / math.sqrt(p.d)
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
            (kc, ks), (vc, vs) = cached_blocks(p, s, b, h // G, "k"), cached_blocks(p, s, b, h // G, "v")
            k, v = kc * ks[:, None], vc * vs[:, None]
            x = q[at:at + n, h].double()
            w = torch.softmax((x @ k.T * sm).masked_fill(~see, -math.inf), -1)
            vv = torch.where(see.any(0)[:, None], v, 0.0)
            o, a = w @ vv, w @ vv.abs()
            # a score's fp32 sum over d products (2^-22 each with the tensor
            # cores' truncation), the query's f16 form (2^-25 of its row's
            # largest), and the three roundings of score + exponent - maximum,
            # an exponent being 40 at most
            size = (x.abs() @ k.abs().T).masked_fill(~see, 0).amax(-1, keepdim=True) * sm
            delta = size * p.d * 2.0 ** -22 + 2.0 ** -17
            delta = delta + 2.0 ** -24 * x.abs().amax(-1, keepdim=True) * k.abs().sum(-1).amax() * sm
            # probabilities to f16: 2^-11, or 2^-25 of a number whose largest, the
            # weight with the value's scale, is 2^7; the result to bf16; fp32 sums
            lost = 2.0 ** -11 + 2 * delta + 2.0 ** -22 * math.sqrt(t)
            most = (w * vs).amax(-1, keepdim=True) * 448
            tol[at:at + n, h] = 2.0 ** -8 * o.abs() + lost * a * 1.01 + t * 2.0 ** -32 * most + 1e-30
            out[at:at + n, h] = o
        at += n
    return out, tol
