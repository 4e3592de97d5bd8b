"""Attention over a cache with block scales on the GPU, both kernels, against
64 bits, and a transformer block's step of all the operators around it."""
import math

import pytest
import torch

import ring_kv_cache_gb300 as kv
from _blockscheck import B, HIGH, LOW, angles_of, attention_blocks_64, cache_of, turned
from _pagescheck import close, errors, i32
from test_gpu_norm import reference as norm_64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

CASES = [
    # hq, hkv, d, page, total, new
    (4, 4, 64, 16, [1], [1]),
    (8, 2, 128, 64, [127, 128, 129, 1, 300], [1, 1, 1, 1, 1]),
    (7, 1, 128, 16, [500, 33, 17], [1, 1, 1]),
    (32, 4, 64, 32, [1000, 77], [2, 0]),
    (10, 10, 128, 128, [2500], [1]),
    (64, 1, 64, 256, [400, 3], [1, 2]),
    (6, 3, 64, 64, [70, 5, 200], [9, 5, 12]),
    (5, 1, 128, 16, [130, 64], [13, 64]),
    (2, 2, 128, 64, [700, 260], [300, 129]),
    (12, 4, 64, 128, [513, 1, 90], [257, 1, 40]),
    (7, 1, 128, 256, [900, 300, 2], [400, 300, 0]),
    (40, 1, 64, 32, [120, 9], [50, 2]),
    (4, 1, 128, 16, [2000], [333]),
]


@pytest.mark.parametrize("mask", ["causal", "window", "all"])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention(case, mask):
    hq, hkv, d, page, total, new = case
    p, s = cache_of(hq, hkv, d, page, total, new, seed=11, layers=2, layer=1, pad=2)
    kw = dict(causal=mask != "all", window=50 if mask == "window" else 0)
    n = sum(new)
    out = torch.full((n + 2, hq, d), 9.0, dtype=BF, device="cuda")
    p.attention(1, s["q"], out=out, **kw)
    want, tol = attention_blocks_64(p, s, **kw)
    close(out[:n], want[:n], tol[:n], mask)
    assert bool((out[n:] == 9.0).all()) and errors(p) == 0
    again = p.attention(1, s["q"], **kw)
    differ = (again[:n] != out[:n]).any(-1).nonzero().tolist()
    assert not differ, ("not the same twice", differ[:8], len(differ))


@pytest.mark.parametrize("total,new,hq,hkv", [([20000], [1], 4, 2), ([9000, 40, 3000, 1, 12000], [1, 1, 1, 1, 1], 8, 8),
                                              ([6000, 100], [40, 30], 8, 1), ([4000], [700], 4, 1), ([9000, 77], [600, 3], 6, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_split_over_many_ranges(total, new, hq, hkv, d):
    p, s = cache_of(hq, hkv, d, 64, total, new, seed=5)
    out = p.attention(0, s["q"])
    want, tol = attention_blocks_64(p, s)
    close(out, want, tol)
    assert errors(p) == 0


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_far_apart(d, new):
    """Values of 2^-38 to 2^38: what carries the result may be the least probable."""
    p, s = cache_of(4, 2, d, 32, [900, 300], [new, new], seed=6, low=-9, high=-4)
    g = torch.Generator(device="cuda").manual_seed(7)
    sc = p.v_scales(0).view(torch.uint8)
    sc.copy_((127 + torch.randint(-38, 39, sc.shape, generator=g, device="cuda")).to(torch.uint8))
    out = p.attention(0, s["q"])
    want, tol = attention_blocks_64(p, s)
    close(out, want, tol)
    # the same for keys: some blocks' scores are large, others' all alike
    ks = p.k_scales(0).view(torch.uint8)
    ks.copy_((127 + torch.randint(-20, 2, ks.shape, generator=g, device="cuda")).to(torch.uint8))
    out = p.attention(0, s["q"])
    want, tol = attention_blocks_64(p, s)
    close(out, want, tol)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("value", [0, 1, 254, 255])
def test_exponents_out_of_range_are_read_as_the_nearest(value, new):
    p, s = cache_of(2, 2, 64, 16, [100], [new], seed=8)
    p.v_scales(0).view(torch.uint8).fill_(value)
    out = p.attention(0, s["q"])
    want, tol = attention_blocks_64(p, s)
    close(out, want, tol)
    p.v_scales(0).view(torch.uint8).fill_(HIGH if value > 100 else LOW)
    assert torch.equal(out, p.attention(0, s["q"]))


@pytest.mark.parametrize("d,new", [(64, 1), (128, 1), (64, 90), (128, 90)])
def test_scores_of_any_size(d, new):
    """Scores beyond 2^20, where the maximum's rounding is wider than the shift; tiny, zero and NaN query rows."""
    p, s = cache_of(2, 1, d, 16, [400], [max(new, 5)], seed=9)
    n = max(new, 5)
    q = s["q"].clone()
    q[0] = 0.0
    q[1] *= 2.0 ** -100
    q[2] *= 2.0 ** 40
    q[3, 0, 0] = math.nan
    q[4] *= 2.0 ** 24
    out = p.attention(0, q)
    want, tol = attention_blocks_64(p, s, q=q)
    ok = [0, 1] + list(range(5, n))
    close(out[ok], want[ok], tol[ok])
    assert bool(torch.isnan(out[3, 0]).all()) and bool(torch.isfinite(out[3, 1]).all())
    for r in (2, 4):   # one-hot on its largest score
        close(out[r], want[r], 2.0 ** -7 * want[r].abs() + 1e-6)
    # scores that differ little beside their size
    p.k_scales(0).view(torch.uint8).fill_(127 + 10)
    c = p.k_cache(0)
    x = torch.full(c.shape, 416.0, device="cuda")
    c.copy_(x.to(c.dtype))
    q = torch.full_like(q, 448.0)
    want, tol = attention_blocks_64(p, s, q=q)
    close(p.attention(0, q), want, tol)


@pytest.mark.parametrize("d,new", [(64, 1), (128, 1), (64, 90), (128, 90)])
def test_the_largest_queries_over_the_largest_scales(d, new):
    """Factors beyond what fp32 holds: one-hot on the largest score, and keys of zeros score 0."""
    p, s = cache_of(2, 1, d, 16, [200], [new], seed=21)
    p.k_scales(0).view(torch.uint8).fill_(HIGH)
    c = p.k_cache(0)
    x = torch.zeros(c.shape, device="cuda")
    page, off = int(p.tables[0, 77 // 16]), 77 % 16
    x[page, 0, off, 3] = 2.0 ** -9
    c.copy_(x.to(c.dtype))
    q = torch.zeros_like(s["q"])
    q[..., 3] = 1.5 * 2.0 ** 127
    q[::2, :, 3] *= -1
    out = p.attention(0, q, causal=False).double()
    at = torch.arange(200, device="cuda")
    ids = p.tables[0, at // 16].long()
    v = p.v_cache(0).view(torch.uint8)[ids, 0, at % 16].view(torch.float8_e4m3fn).double()
    v = v * torch.exp2(p.v_scales(0).view(torch.uint8)[ids, 0, 0].double() - 127)[:, None]
    others = torch.cat([v[:77], v[78:]]).mean(0)
    for t in range(new):   # (the fp32 sum of 199 values and f16 probabilities: 2^-10 of their sizes)
        want = others if t % 2 == 0 else v[77]
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -10 * v.abs().mean(0) if t % 2 == 0 else 0)
        close(out[t], want.expand(2, -1), tol.expand(2, -1))


@pytest.mark.parametrize("rise", [0.03, 0.4, 3.0])
@pytest.mark.parametrize("d,new", [(128, 1), (128, 70), (64, 3), (64, 200)])
def test_scores_that_keep_rising(d, new, rise):
    """Scores that grow by `rise` (log2 units) a token: running maxima that are raised never, now and then or by every tile."""
    total = 900
    p, s = cache_of(2, 2, d, 32, [total], [new], seed=14)
    c, ks = p.k_cache(0), p.k_scales(0).view(torch.uint8)
    ks.fill_(120)
    at = torch.arange(total, device="cuda")
    pages, off = p.tables[0, at // 32].long(), at % 32
    x = c.float()
    x[..., 0] = 0.0
    x[pages, :, off, 0] = (at * (440.0 / total))[:, None].expand(total, 2)
    c.copy_(x.to(c.dtype))
    q = 0.05 * s["q"].float()
    q[..., 0] = rise * total / 440.0 / (2.0 ** -7 * math.log2(math.e) / math.sqrt(d))
    q = q.to(BF)
    want, tol = attention_blocks_64(p, s, q=q)
    close(p.attention(0, q), want, tol)
    assert errors(p) == 0


@pytest.mark.parametrize("d,hq,hkv,total,new,bad,window", [
    (128, 4, 2, [300, 90], [5, 1], 297, 0), (64, 4, 4, [300, 90], [8, 1], 295, 0), (64, 12, 4, [400], [6], 197, 200),
    (128, 4, 2, [300, 90], [200, 3], 250, 0), (64, 2, 1, [700], [300], 650, 0), (64, 2, 2, [900], [400], 350, 200)])
def test_hidden_values_reach_no_row(d, hq, hkv, total, new, bad, window):
    """A key and a value of one token are NaN: the rows whose mask hides it are as if it were not there."""
    p, s = cache_of(hq, hkv, d, 32, total, new, seed=12)
    page, off = int(p.tables[0, bad // 32]), bad % 32
    clean, tol = attention_blocks_64(p, s, window=window)
    p.k_cache(0)[page, :, off] = math.nan
    p.v_cache(0)[page, :, off] = math.nan
    out = p.attention(0, s["q"], window=window)
    pos = torch.arange(total[0] - new[0], total[0], device="cuda")
    sees = (pos >= bad) & ((pos - window < bad) if window else True)
    sees = torch.cat([sees, torch.zeros(sum(new[1:]), dtype=torch.bool, device="cuda")])
    n = sum(new)
    close(out[:n][~sees], clean[:n][~sees], tol[:n][~sees])
    assert bool(torch.isnan(out[:n][sees]).all())


def test_pages_that_are_none_read_as_zeros():
    p, s = cache_of(2, 1, 64, 16, [50, 200], [1, 60], seed=13, missing={(0, 1), (1, 3)})
    s["q"][:] = 0.0     # every token alike
    out = p.attention(0, s["q"])
    want = torch.zeros(61, 64, dtype=torch.float64, device="cuda")
    at = 0
    for b, (t, n) in enumerate(zip(s["total"], s["new"])):
        v = torch.zeros((t, 64), dtype=torch.float64, device="cuda")
        for j in range(t):
            page = int(p.tables[b, j // 16])
            if 0 <= page < p.num_pages:
                e = p.v_scales(0).view(torch.uint8)[page, 0, 0].item()
                v[j] = p.v_cache(0)[page, 0, j % 16].double() * 2.0 ** (min(max(e, LOW), HIGH) - 127)
        for i in range(n):
            want[at + i] = v[:t - n + i + 1].mean(0)
        at += n
    close(out, want[:, None].expand(-1, 2, -1), 2.0 ** -7 * want.abs()[:, None] + 1e-3)
    assert errors(p) & kv.PAGES_ERR_TABLE


def test_strided_queries_and_tensors_shorter_than_the_plan():
    p, s = cache_of(4, 2, 128, 64, [300, 150], [3, 5], seed=16)
    wide = torch.randn((8, 9, 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(BF)
    q = wide[:, 3:7]
    want, tol = attention_blocks_64(p, s, q=q, scale=0.3)
    close(p.attention(0, q, scale=0.3), want, tol)
    for n in (1, 3, 6):
        close(p.attention(0, q[:n], scale=0.3), want[:n], tol[:n], n)


@pytest.mark.parametrize("new", [1, 300])
def test_waits_that_give_up(new):
    p, s = cache_of(4, 2, 128, 64, [500], [new], seed=17)
    want = p.attention(0, s["q"])
    torch.cuda.synchronize()
    p.set_wait(2_000_000, True)
    p.attention(0, s["q"])
    torch.cuda.synchronize()
    assert errors(p) == kv.PAGES_ERR_TIMEOUT
    p.set_wait()
    p.state[kv.PAGES_STATE["error"]] = 0
    p.plan(i32([new]), new)
    assert torch.equal(p.attention(0, s["q"]), want) and errors(p) == 0


def test_two_caches_on_two_streams():
    a, sa = cache_of(8, 2, 128, 64, [3000, 700], [1, 200], seed=18)
    b, sb = cache_of(8, 8, 64, 16, [2000, 900], [1, 300], seed=19)
    want = [a.attention(0, sa["q"]), b.attention(0, sb["q"])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        x = a.attention(0, sa["q"])
        y = b.attention(0, sb["q"], stream=side)
        torch.cuda.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])


# ------------------------------------------------------- a block's step
@pytest.mark.parametrize("hq,hkv,d,norm", [(4, 4, 128, "layer"), (8, 2, 64, "rms")])
def test_a_transformer_blocks_step(hq, hkv, d, norm):
    """Norm and modulation, projection, write by (t, y, x) into blocks, attention,
    projection, gate and the next norm: two requests over three steps, every
    link against 64 bits from its own inputs, then the same steps in a graph."""
    D, steps, rows = hq * d, 3, 8
    new = [21, 6]
    n = sum(new)
    rope3d = (d // 4, d // 8)
    g = torch.Generator(device="cuda").manual_seed(20)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    w_in = (rand((hq + 2 * hkv) * d, D) / math.sqrt(D)).to(BF)
    w_out = (rand(D, hq * d) / math.sqrt(hq * d)).to(BF)
    wq, wk = [(1 + 0.2 * rand(d)).to(BF) for _ in "qk"]
    mod = 0.3 * rand(2, 5, D)           # scale, shift of the attention's norm; its gate; scale, shift of the next
    idx = i32([0] * new[0] + [1] * new[1])
    stream0, xyz = rand(n, D), torch.randint(0, 50, (n, 3), generator=g, device="cuda").to(torch.int32)
    count = i32(new)

    def cache():
        return kv.KvPages(hq, hkv, d, page_size=16, num_pages=40, max_requests=2, max_request_tokens=16 * rows, max_tokens=n,
                          block_scales=True, rope3d=rope3d, max_position=50)

    def step(p, h):
        x = kv.residual_norm(h, norm=norm, scale=mod[:, 0], shift=mod[:, 1], mod_rows=idx)[1]
        qkv = (x @ w_in.t()).view(n, hq + 2 * hkv, d)
        q, k, v = qkv.split([hq, hkv, hkv], dim=1)
        p.plan(count, n)
        qr = p.write(0, q, k, v, q_norm=wq, k_norm=wk, pos=xyz)
        o = p.attention(0, qr, causal=False)
        y = o.view(n, D) @ w_out.t()
        h2, x2 = kv.residual_norm(h, y, gate=mod[:, 2], norm=norm, scale=mod[:, 3], shift=mod[:, 4], mod_rows=idx, residual_scale=0.5)
        p.commit()
        return x, qkv, qr, o, y, h2, x2

    p, h, done = cache(), stream0, []
    for i in range(steps):
        x, qkv, qr, o, y, h2, x2 = step(p, h)
        total = [(i + 1) * c for c in new]
        s = dict(total=total, new=new, layer=0)
        _, (want, tol) = norm_64(dict(h=h, mod=torch.stack([mod[:, 2], mod[:, 0], mod[:, 1]], 1)), idx=idx, norm=norm, y=False)
        close(x, want, tol, "first norm")
        want, m = turned(qkv[:, :hq], wq, angles_of(d, xyz, rope3d), "adjacent")
        close(qr, want, 2.0 ** -8 * want.abs() + 2.0 ** -19 * m + 1e-30, "queries")
        keys = turned(qkv[:, hq:hq + hkv], wk, angles_of(d, xyz, rope3d), "adjacent")[0]
        sl = p._slots[:n].long()
        sc = torch.exp2(p.k_scales(0).view(torch.uint8)[sl // 16, :, sl % 16 // B].double() - 127)
        got = p.k_cache(0).view(torch.uint8)[sl // 16, :, sl % 16].view(torch.float8_e4m3fn).double() * sc[..., None]
        close(got, keys, 2.0 ** -4 * keys.abs() + 2.0 ** -9 * sc[..., None] + 2.0 ** -18, "keys")
        want, tol = attention_blocks_64(p, s, q=qr, causal=False)
        close(o, want, tol, "attention")
        (hw, th), (xw, tx) = norm_64(dict(h=h, y=y, mod=mod[:, 2:]), alpha=0.5, idx=idx, norm=norm)
        close(h2, hw, th, "stream")
        close(x2, xw, tx, "next norm")
        h = h2
        done.append((o, h2, x2))
    assert errors(p) == 0 and p.lengths.tolist() == [steps * c for c in new]
    # the same in a graph, each replay a step
    r, h = cache(), stream0.clone()
    step(r, h)
    r.release(i32([0, 1]))
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        _, _, _, o, _, h2, x2 = step(r, h)
        h.copy_(h2)
    for i in range(steps):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip((o, h2, x2), done[i])), i
