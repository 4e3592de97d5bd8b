"""The paged cache on the GPU against plain 64-bit forms: plan, commit and
release against a host allocator, the write, the attention, and steps of
all of them together."""
import math
import random

import pytest
import torch

import ring_kv_cache_gb300 as kv
from _pagescheck import Allocator, attention_64, close, errors, filled, i32, norm_rope_64

pytestmark = pytest.mark.gpu


def pool(page=16, num_pages=40, rows=6, most=200, tokens=64, **kw):
    return kv.KvPages(kw.pop("hq", 2), kw.pop("hkv", 1), kw.pop("d", 64), page_size=page, num_pages=num_pages,
                      max_requests=rows, max_request_tokens=most, max_tokens=tokens, **kw)


def check_state(p, a):
    torch.cuda.synchronize()
    assert p.lengths.tolist() == a.lens
    n = p.state[kv.PAGES_STATE["free"]].item()
    assert p.free_pages[:n].tolist() == a.free
    tab = p.tables.tolist()
    for r, ln in enumerate(a.lens):
        w = -(-ln // a.page)
        assert tab[r][:w] == a.table[r][:w], r


# ------------------------------------------------------------------- plan
@pytest.mark.parametrize("page,rows,tokens,seed", [(16, 6, 64, 0), (64, 33, 500, 1), (128, 5, 3000, 2), (256, 3, 700, 3),
                                                   (16, 700, 5000, 4), (32, 1, 1, 5), (16, 1500, 2049, 6)])
def test_steps_follow_a_host_allocator(page, rows, tokens, seed):
    rng = random.Random(seed)
    most = max(3 * page + 5, 4 * tokens // rows + 40)
    num = max(4, rows * 2 + tokens // page)
    p = pool(page, num, rows, most, tokens)
    a = Allocator(rows, p.W, page, num)
    for step in range(12):
        n = rng.randint(1, rows)
        which = rng.sample(range(rows), n)
        left, new = tokens, []
        for _ in which:
            x = rng.choice([0, 1, 1, 2, rng.randint(0, max(1, 3 * tokens // n))])
            new.append(min(left, x))
            left -= new[-1]
        want = a.plan(which, new, tokens)
        got = p.plan(i32(new), tokens, rows=i32(which), max_new=max(1, max(new)))
        if want is None:   # no room: refused, and end some requests
            assert errors(p) & (kv.PAGES_ERR_PAGES | kv.PAGES_ERR_LENGTH)
            assert got.cu.tolist() == [0] * (n + 1) and set(got.slots.tolist()) == {-1}
            p.state[kv.PAGES_STATE["error"]] = 0
            p.commit()
            check_state(p, a)
            done = rng.sample(range(rows), max(1, rows // 2))
            p.release(i32(done))
            a.release(done)
        else:
            cu, lens, pos, slots, fresh, taken = want
            assert got.cu.tolist() == cu and got.lengths.tolist() == lens
            assert got.positions.tolist() == pos and got.slots.tolist() == slots
            assert p.state[kv.PAGES_STATE["taken"]].item() == taken
            if rng.random() < 0.7:   # a plan that is not committed costs nothing
                p.commit()
                a.commit(which, want)
        check_state(p, a)
    assert errors(p) == 0


@pytest.mark.parametrize("rows,new,tokens,max_new,bit", [
    ([0, 0], [1, 1], 8, None, kv.PAGES_ERR_ROW), ([0, 6], [1, 1], 8, None, kv.PAGES_ERR_ROW),
    ([-1, 2], [1, 1], 8, None, kv.PAGES_ERR_ROW), ([0, 1], [1, -1], 8, None, kv.PAGES_ERR_TOKENS),
    ([0, 1], [5, 4], 8, None, kv.PAGES_ERR_TOKENS), ([0, 1], [5, 1], 8, 4, kv.PAGES_ERR_TOKENS),
    ([0, 1], [2 ** 31 - 1, 2 ** 31 - 1], 8, None, kv.PAGES_ERR_TOKENS), ([4, 1], [30, 2], 64, None, kv.PAGES_ERR_LENGTH),
    ([0, 1], [50, 14], 64, None, kv.PAGES_ERR_PAGES)])
def test_plans_that_cannot_be_made(rows, new, tokens, max_new, bit):
    p = pool(16, 4, 6, 64, 64)
    p.restore(i32([0, 0, 0, 0, 40, 0]), torch.full((6, 4), -1, dtype=torch.int32, device="cuda"), i32([0, 1, 2, 3]))
    step = p.plan(i32(new), tokens, rows=i32(rows), max_new=max_new)
    assert errors(p) == bit
    assert step.cu.tolist() == [0, 0, 0] and step.slots.tolist() == [-1] * tokens
    p.commit()
    assert p.lengths.tolist() == [0, 0, 0, 0, 40, 0] and p.state[kv.PAGES_STATE["free"]].item() == 4
    q = torch.ones((tokens, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 3.0)
    p.attention(0, q, out=out)   # nothing planned: nothing written
    assert bool((out == 3.0).all())


def test_pages_that_the_pool_does_not_have_are_reported_and_skipped():
    p = pool(16, 4, 2, 64, 64, cache_dtype=torch.bfloat16)
    p.restore(i32([20, 5]), i32([[0, 99, -1, -1], [-7, -1, -1, -1]]), i32([1, 77]))
    step = p.plan(i32([3, 14]), 20)
    # request 0: page id 99; request 1: -7, then from the free list 77
    assert step.slots.tolist() == [-1] * 20
    assert errors(p) == kv.PAGES_ERR_TABLE
    q = torch.ones((20, 2, 64), dtype=torch.bfloat16, device="cuda")
    p.k_cache(0).fill_(1.0)
    p.v_cache(0).fill_(1.0)
    k = torch.ones((20, 1, 64), dtype=torch.bfloat16, device="cuda")
    p.write(0, q, k, k * 5)
    out = p.attention(0, q)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out[:17]).all()) and bool((p.v_cache(0) == 1.0).all())


def test_commit_and_release_refusals():
    p = pool(16, 8, 4, 64, 64)
    p.commit()
    assert errors(p) == kv.PAGES_ERR_COMMIT
    p.state[kv.PAGES_STATE["error"]] = 0
    p.plan(i32([20, 3]), 23)
    p.commit()
    for bad in ([0, 0], [0, 4], [-1]):
        p.release(i32(bad))
        assert errors(p) == kv.PAGES_ERR_ROW
        p.state[kv.PAGES_STATE["error"]] = 0
        assert p.lengths.tolist() == [20, 3, 0, 0] and p.state[kv.PAGES_STATE["free"]].item() == 5
    p.release(i32([1, 3]))   # an empty row is no error
    assert errors(p) == 0 and p.lengths.tolist() == [20, 0, 0, 0] and p.state[kv.PAGES_STATE["free"]].item() == 6
    p.plan(i32([1]), 1)
    p.release(i32([0]))      # drops the plan
    p.commit()
    assert errors(p) == kv.PAGES_ERR_COMMIT and p.lengths.tolist() == [0, 0, 0, 0]
    assert sorted(p.free_pages.tolist()) == list(range(8))


# ------------------------------------------------------------------ write
def check_write(p, s, qkv, norm, pairing, tokens, wq, wk, eps=1e-6):
    hq, hkv, d = p.Hq, p.Hkv, p.d
    n = qkv.shape[0]
    q, k, v = qkv.view(n, hq + 2 * hkv, d).split([hq, hkv, hkv], dim=1)
    before_k, before_v = p.k_cache(s["layer"]).clone(), p.v_cache(s["layer"]).clone()
    q_out = torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    p.write(s["layer"], q, k, v, q_norm=wq, k_norm=wk, eps=eps, q_out=q_out)
    torch.cuda.synchronize()
    assert bool((q_out[tokens:] == 7.0).all()), "rows past the plan"
    pos, slots = p._pos[:tokens].long(), p._slots[:tokens].long()
    fp = 2.0 ** -19   # fp32: the sum over d, rsqrt, the products
    want, m = norm_rope_64(q[:tokens], wq, pos, pairing, eps)
    close(q_out[:tokens], want, 2.0 ** -8 * want.abs() + fp * m + 1e-30, "q")
    e4m3 = p.cache_dtype == torch.float8_e4m3fn
    for name, x, w, cache, before in (("k", k, wk, p.k_cache(s["layer"]), before_k),
                                      ("v", v, None, p.v_cache(s["layer"]), before_v)):
        want, m = norm_rope_64(x[:tokens], w, pos if name == "k" else None, pairing, eps)
        raw = cache.view(torch.uint8) if e4m3 else cache
        got = raw[slots // p.P, :, slots % p.P]
        if e4m3:
            sc = s["s" + name].double()[:, None]
            want, m = want / sc, m / sc
            tol = 2.0 ** -4 * want.abs() + 2.0 ** -10 + fp * m
            want = want.clamp(-448, 448)
            got = got.view(cache.dtype)
        else:
            tol = (2.0 ** -8 * want.abs() + fp * m) * (1 if name == "k" else 0)
        close(got.to(torch.float64), want, tol + 1e-30, name)
        # nothing else has changed
        other = torch.ones((p.num_pages, p.P), dtype=torch.bool, device="cuda")
        other[slots // p.P, slots % p.P] = False
        a, b = [t.view(torch.uint8).view(p.num_pages, hkv, p.P, -1).transpose(1, 2)[other] for t in (cache, before)]
        assert torch.equal(a, b), name


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,page,total,new,pad", [
    (4, 2, 64, 16, [37, 1, 64, 20], [3, 1, 0, 17], 5), (10, 10, 128, 64, [1], [1], 0), (7, 1, 128, 128, [300, 129], [150, 1], 1),
    (40, 8, 64, 256, [700], [500], 0), (3, 3, 64, 32, [33] * 9, [1] * 9, 3)])
def test_write(hq, hkv, d, page, total, new, pad, cache, pairing):
    p, s = filled(hq, hkv, d, page, total, new, cache, seed=1, layers=2, layer=1, pairing=pairing, pad=pad)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    n = sum(new) + pad
    for norm in (True, False):
        qkv = (3.0 * torch.randn((n, (hq + 2 * hkv) * d), generator=g, device="cuda")).to(torch.bfloat16)
        qkv[sum(new):] = math.nan   # padding is not read
        wq, wk = [(0.5 + torch.rand(d, generator=g, device="cuda")).to(torch.bfloat16) if norm else None for _ in "qk"]
        check_write(p, s, qkv, norm, pairing, sum(new), wq, wk)
    assert errors(p) == 0


def test_write_extremes():
    """Zero rows, saturation, infinities and NaN stay in their own rows."""
    p, s = filled(2, 2, 64, 16, [8], [8], "e4m3", seed=3)
    x = torch.ones((8, 6, 64), dtype=torch.bfloat16, device="cuda")
    x[0] = 0.0
    x[1] = 3e38
    x[2, :, 5] = math.inf
    x[3, :, 9] = math.nan
    q, k, v = x.split([2, 2, 2], dim=1)
    one = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    q_out = p.write(0, q, k, v, q_norm=one, k_norm=one)
    sl = p._slots[:8].long()
    kc = p.k_cache(0).view(torch.uint8)[sl // 16, :, sl % 16].view(torch.float8_e4m3fn).float()
    vc = p.v_cache(0).view(torch.uint8)[sl // 16, :, sl % 16].view(torch.float8_e4m3fn).float()
    assert bool((q_out[0] == 0).all()) and bool((kc[0] == 0).all()) and bool((vc[0] == 0).all())
    assert bool((vc[1] == 448).all())
    assert bool((vc[2, :, 5] == 448).all()) and bool(torch.isnan(vc[3, :, 9]).all())
    for t in (4, 5, 6, 7):
        assert bool(torch.isfinite(q_out[t]).all()) and bool(torch.isfinite(kc[t]).all())
    assert bool(torch.isnan(q_out[3]).all())


# -------------------------------------------------------------- attention
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
@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention(case, cache, mask):
    hq, hkv, d, page, total, new = case
    p, s = filled(hq, hkv, d, page, total, new, cache, seed=11, layers=2, layer=1, pad=2)
    kw = dict(causal=mask != "all", window=50 if mask == "window" else 0)
    n = sum(new)
    out = torch.full((n + 2, hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    p.attention(1, s["q"], out=out, **kw)
    want, tol = attention_64(p, s, **kw)
    close(out[:n], want[:n], tol[:n], mask)
    assert bool((out[n:] == 9.0).all()) and errors(p) == 0
    again = p.attention(1, s["q"], **kw)
    differ = (again[:n] != out[:n]).any(-1).nonzero().tolist()
    assert not differ, ("not the same twice", differ[:8], len(differ))


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("total,new,hq,hkv", [([20000], [1], 4, 2), ([9000, 40, 3000, 1, 12000], [1, 1, 1, 1, 1], 8, 8),
                                              ([6000, 100], [40, 30], 8, 1), ([4000], [700], 4, 1)])
def test_attention_split_over_many_ranges(total, new, hq, hkv, cache):
    p, s = filled(hq, hkv, 128, 64, total, new, cache, seed=5)
    out = p.attention(0, s["q"])
    want, tol = attention_64(p, s)
    close(out, want, tol)
    assert errors(p) == 0


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_attention_strided_queries_scale_and_large_scores(cache):
    p, s = filled(4, 2, 128, 64, [300, 150], [1, 5], cache, seed=6, magnitude=40.0)
    wide = torch.randn((6, 9, 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.bfloat16)
    q = wide[:, 3:7]
    assert not q.is_contiguous()
    out = p.attention(0, q, scale=0.3)
    want, tol = attention_64(p, s, q=q, scale=0.3)
    close(out, want, tol)


def test_tensors_shorter_than_the_plan():
    """The planned tokens that the tensors hold, at their own positions."""
    p, s = filled(4, 2, 64, 16, [40, 30, 9], [3, 5, 4], "bf16", seed=8)
    want, tol = attention_64(p, s)
    for n in (1, 3, 6, 8, 11):
        out = p.attention(0, s["q"][:n])
        close(out, want[:n], tol[:n], n)


@pytest.mark.parametrize("new", [5, 90])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_queries_of_any_size(cache, d, new):
    """Tiny, zero and huge query rows: the 8-bit cache's queries change type."""
    p, s = filled(2, 1, d, 16, [300], [new], cache, seed=7)
    q = s["q"].clone()
    q[0] = 0.0
    q[1] *= 2.0 ** -100
    q[2] *= 2.0 ** 40
    q[3, 0, 0] = math.nan
    out = p.attention(0, q)
    want, tol = attention_64(p, s, q=q)
    ok = [0, 1, 4] + list(range(5, new))
    close(out[ok], want[ok], tol[ok])
    assert bool(torch.isnan(out[3, 0]).all()) and bool(torch.isfinite(out[3, 1]).all())
    # row 2 is one-hot on its largest score
    close(out[2], want[2], 2.0 ** -7 * want[2].abs() + 1e-6)


@pytest.mark.parametrize("rise", [0.03, 0.4, 3.0])
@pytest.mark.parametrize("d,new", [(128, 1), (128, 70), (64, 3), (64, 200)])
@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_scores_that_keep_rising(cache, d, new, rise):
    """Scores that grow by `rise` (log2 units) a token: running maxima that
    are raised never, now and then or by every tile."""
    total = 900
    p, s = filled(2, 2, d, 32, [total], [new], cache, seed=14)
    c = p.k_cache(0)
    up = torch.arange(total, device="cuda") * (440.0 / total)
    pages, off = p.tables[0, torch.arange(total, device="cuda") // 32].long(), torch.arange(total, device="cuda") % 32
    x = c.float()
    x[..., 0] = 0.0
    x[pages, :, off, 0] = up[:, None].expand(total, 2)
    c.copy_(x.to(c.dtype))
    q = 0.05 * s["q"].float()
    scale = s["sk"] if cache == "e4m3" else torch.ones(2, device="cuda")
    q[..., 0] = rise * total / 440.0 / (scale * math.log2(math.e) / math.sqrt(d))
    q = q.to(torch.bfloat16)
    want, tol = attention_64(p, s, q=q)
    close(p.attention(0, q), want, tol)
    assert errors(p) == 0


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("d,hq,hkv,total,new,bad,window", [
    (128, 4, 2, [300, 90], [5, 1], 297, 0), (64, 4, 4, [300, 90], [8, 1], 295, 0), (64, 12, 4, [400], [6], 197, 200),
    (128, 4, 2, [300, 90], [200, 3], 250, 0), (64, 2, 1, [700], [300], 650, 0), (64, 2, 2, [900], [400], 350, 200),
    (128, 5, 1, [400], [100], 390, 0)])
def test_hidden_values_reach_no_row(d, hq, hkv, total, new, bad, window, cache, value):
    """A key and a value of one token are not finite: the rows whose mask
    hides it are as if it were not there, the others are not finite."""
    if cache == "e4m3":
        value = math.nan   # E4M3 has no infinities
    p, s = filled(hq, hkv, d, 32, total, new, cache, seed=12)
    page, off = int(p.tables[0, bad // 32]), bad % 32
    want, tol = attention_64(p, s, window=window)
    pos = torch.arange(total[0] - new[0], total[0], device="cuda")
    sees = (pos >= bad) & ((pos < bad + window) if window else True)
    assert bool(sees.any()) and not bool(sees.all())
    c = p.v_cache(0)
    for key in (False, True):
        c = p.k_cache(0) if key else p.v_cache(0)
        before = c[page, :, off].clone()
        row = before.float()
        row[:, 3] = value
        c[page, :, off] = row.to(c.dtype)
        out = p.attention(0, s["q"], window=window)
        n = new[0]
        close(out[:n][~sees], want[:n][~sees], tol[:n][~sees], "hidden")
        close(out[n:], want[n:], tol[n:], "other requests")
        if not key:
            o = out[:n][sees]
            assert not bool(torch.isfinite(o[..., 3]).any())
            rest = [i for i in range(d) if i != 3]
            close(o[..., rest], want[:n][sees][..., rest], tol[:n][sees][..., rest], "its other columns")
            if value == math.inf:
                assert bool((o[..., 3] == math.inf).all())
        elif math.isnan(value):
            assert bool(torch.isnan(out[:n][sees]).all())
        c[page, :, off] = before
    assert errors(p) == 0


@pytest.mark.parametrize("new", [1, 60])
def test_large_values_and_tiny_scales(new):
    """bf16 values near the end of their range, and scales that leave no score."""
    p, s = filled(4, 2, 128, 64, [300], [new], "bf16", seed=13)
    p.v_cache(0).mul_(2.0 ** 114)
    want, tol = attention_64(p, s)
    out = p.attention(0, s["q"])
    close(out, want, tol)
    p.v_cache(0).mul_(2.0 ** -114)
    for cache in ("bf16", "e4m3"):
        p, s = filled(4, 2, 128, 64, [300], [new], cache, seed=13)
        for scale in (1e-44, 1e-30):
            out = p.attention(0, s["q"], scale=scale)
            want, tol = attention_64(p, s, scale=scale)
            close(out, want, tol)
    with pytest.raises(kv.KvRingError):
        p.attention(0, s["q"], scale=3e38)


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
def test_a_cache_beyond_32_bit_offsets(cache):
    """Pages whose bytes lie beyond 2^32 of the pool, in a later layer."""
    hq, hkv, d, page, num = 8, 8, 128, 64, 24000 if cache == "bf16" else 40000
    dt = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    p = kv.KvPages(hq, hkv, d, page_size=page, num_pages=num, max_requests=2, max_request_tokens=6 * page,
                   max_tokens=200, layers=2, cache_dtype=dt)
    assert p.k_cache(1)[num - 9].data_ptr() - p.k_cache(0).data_ptr() > 2 ** 32
    ids = torch.full((2, 6), -1, dtype=torch.int32, device="cuda")
    ids[0, :3] = torch.tensor([num - 1, 0, num - 2], dtype=torch.int32)
    ids[1, :2] = torch.tensor([num - 5, num - 9], dtype=torch.int32)
    p.restore(i32([150, 100]), ids, i32([1, num - 3, num - 4, num - 6]))
    g = torch.Generator(device="cuda").manual_seed(4)
    for c in (p.k_cache(1), p.v_cache(1)):
        for i in (num - 1, 0, num - 2, num - 5, num - 9):
            c[i] = torch.randn(c.shape[1:], generator=g, device="cuda").to(dt)
    s = dict(layer=1)
    if cache == "e4m3":
        s.update(sk=torch.ones(hkv, device="cuda"), sv=torch.ones(hkv, device="cuda"))
    for new in ([1, 1], [120, 70]):
        n = sum(new)
        p.plan(i32(new), n, max_new=max(new))
        qkv = torch.randn((n, 3 * hq, d), generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = qkv.split([hq, hkv, hkv], dim=1)
        q_out = p.write(1, q, k, v)
        out = p.attention(1, q_out)
        s.update(total=[150 + new[0], 100 + new[1]], new=new, before=[150, 100])
        want, tol = attention_64(p, s, q=q_out)
        close(out, want, tol)
        # the values written are those read back
        sl = p._slots[:n].long()
        raw = p.v_cache(1).view(torch.uint8)[sl // page, :, sl % page] if cache == "e4m3" else \
            p.v_cache(1)[sl // page, :, sl % page]
        got = raw.view(dt).float()
        close(got, v.double(), (2.0 ** -4 * v.double().abs() + 2.0 ** -10) if cache == "e4m3" else 0 * v.double(), "v")
    assert errors(p) == 0


def test_two_caches_on_two_streams_at_once():
    """Objects of their own are independent: chunks on one stream, single
    tokens on another, and a ring's projection feeding the pages."""
    a, sa = filled(4, 2, 128, 64, [3000, 700], [500, 200], "bf16", seed=20)
    b, sb = filled(8, 8, 64, 16, [5000, 80, 900], [1, 1, 1], "e4m3", seed=21)
    wa, ta = attention_64(a, sa)
    wb, tb = attention_64(b, sb)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(torch.zeros_like(sa["q"]), torch.zeros_like(sb["q"])) for _ in range(6)]
    torch.cuda.synchronize()
    for oa, ob in outs:
        a.attention(0, sa["q"], out=oa, stream=s1)
        b.attention(0, sb["q"], out=ob, stream=s2)
    torch.cuda.synchronize()
    for oa, ob in outs:
        close(oa, wa, ta, "a")
        close(ob, wb, tb, "b")


def test_the_rings_projection_feeds_the_pages():
    """Queries, keys and values from kvring_project_write, read by the write
    right behind it, and the pages' output read by a ring's write."""
    H, d, n, dm = 2, 64, 12, 128
    ring = kv.KvRing(H, d, 48, n, 256)
    p = kv.KvPages(H, H, d, page_size=16, num_pages=20, max_requests=1, max_request_tokens=300, max_tokens=n,
                   cache_dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(5)
    w = (0.1 * torch.randn((3 * H * d, dm), generator=g, device="cuda")).to(torch.bfloat16)
    xs = [torch.randn((n, dm), generator=g, device="cuda").to(torch.bfloat16) for _ in range(8)]
    ones = torch.ones((n, H, d), dtype=torch.bfloat16, device="cuda")
    ring.calibrate(ones, ones)
    torch.cuda.synchronize()
    got, kept = [], []
    for x in xs:
        q, kv_out = ring.project_write(x, w, write=False, store_kv=True)
        p.plan(i32([n]), n)
        q_out = p.write(0, q, kv_out[0], kv_out[1])
        out = p.attention(0, q_out)
        p.commit()
        ring.write(out, out)   # reads the pages' output
        got.append(out)
        kept.append((q, kv_out))
    e = ring.export()
    torch.cuda.synchronize()
    total = n * len(xs)
    s = dict(total=[total], new=[n], before=[total - n], layer=0)
    p.plan(i32([0]), n)
    for i, (q, kv_out) in enumerate(kept):
        pos = torch.arange(i * n, (i + 1) * n, device="cuda")
        q_want = norm_rope_64(q, None, pos, "adjacent")[0].to(torch.bfloat16)
        s.update(total=[(i + 1) * n])
        want, tol = attention_64(p, s, q=q_want)
        # (a rotated query may have been rounded the other way)
        close(got[i], want, tol + 2.0 ** -6 * want.abs().amax(), i)
    last = torch.cat(got[-4:]).float()          # the ring's 48 slots: the last four outputs
    codes = e["v"].view(torch.float8_e4m3fn).float() * e["scales"][H:2 * H, None, None]
    order = torch.argsort(e["slot_pos"])
    close(codes[:, order].transpose(0, 1), last.clamp(-1, 1).double(), 2.0 ** -4 * last.abs() + 2.0 ** -10, "ring")


# --------------------------------------------------------------- together
def plain_step(hist, qkv, cu, hq, hkv, d, pairing, wq, wk, cache, sk, sv):
    """One layer's step on host lists of (k, v) float64 per request."""
    q, k, v = qkv.view(-1, hq + 2 * hkv, d).split([hq, hkv, hkv], dim=1)
    outs = []
    for r, (a, b) in hist["span"].items():
        n = b - a
        pos = torch.arange(hist["len"][r], hist["len"][r] + n, device="cuda")
        qq = norm_rope_64(q[a:b], wq, pos, pairing)[0].to(torch.bfloat16).double()
        kk, vv = norm_rope_64(k[a:b], wk, pos, pairing)[0], v[a:b].double()
        if cache == "e4m3":
            rnd = lambda x, sc: ((x / sc[:, None].double()).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()  # noqa: E731
                                 * sc[:, None].double())
            kk, vv = rnd(kk, sk), rnd(vv, sv)
        else:
            kk = kk.to(torch.bfloat16).double()
        old = hist["kv"].get(r)
        kk, vv = (kk, vv) if old is None else (torch.cat([old[0], kk]), torch.cat([old[1], vv]))
        hist["kv"][r] = (kk, vv)
        G = hq // hkv
        w = torch.einsum("ihd,jhd->hij", qq, kk.repeat_interleave(G, 1)) / math.sqrt(d)
        j = torch.arange(kk.shape[0], device="cuda")
        w = torch.softmax(w.masked_fill(j[None, None] > pos[None, :, None], -math.inf), -1)
        outs.append((r, torch.einsum("hij,jhd->ihd", w, vv.repeat_interleave(G, 1))))
    return dict(outs)


@pytest.mark.parametrize("cache,pairing,graph", [("bf16", "halves", False), ("e4m3", "adjacent", False),
                                                 ("e4m3", "halves", True)])
def test_steps_of_all_operators_together(cache, pairing, graph):
    """Prompts, single tokens, ended and restarted requests, as a serving
    loop runs them; decode steps captured once and replayed."""
    hq, hkv, d, rows = 6, 2, 64, 5
    dt = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
    p = kv.KvPages(hq, hkv, d, page_size=16, num_pages=60, max_requests=rows, max_request_tokens=300, max_tokens=260,
                   cache_dtype=dt, rope_pairing=pairing)
    g = torch.Generator(device="cuda").manual_seed(3)
    sk, sv = torch.full((hkv,), 0.02, device="cuda"), torch.full((hkv,), 0.01, device="cuda")
    if cache == "e4m3":
        p.set_scales(0, sk, sv)
    wq, wk = [(0.8 + 0.4 * torch.rand(d, generator=g, device="cuda")).to(torch.bfloat16) for _ in "qk"]
    hist = dict(len=[0] * rows, kv={}, span={})
    decode = {}

    def run(qkv, q_out, out):
        q, k, v = qkv.view(-1, hq + 2 * hkv, d).split([hq, hkv, hkv], dim=1)
        p.write(0, q, k, v, q_norm=wq, k_norm=wk, q_out=q_out)
        p.attention(0, q_out, out=out)
        p.commit()

    plan = [([0, 1, 2], [130, 7, 40]), ([2, 0, 1], [1, 1, 1]), ([0, 1, 2], [1, 1, 1]), ([0, 1, 2], [1, 1, 1]), "end 0",
            ([0, 3, 1], [33, 64, 1]), ([1, 3, 0], [1, 1, 1]), ([0, 4, 2, 3], [3, 90, 0, 1])]
    for step in plan:
        if step == "end 0":
            p.release(i32([0]))
            hist["len"][0] = 0
            del hist["kv"][0]
            continue
        which, new = step
        n = sum(new)
        qkv = (2 * torch.randn((n, (hq + 2 * hkv) * d), generator=g, device="cuda")).to(torch.bfloat16)
        hist["span"], at = {}, 0
        for r, m in zip(which, new):
            if m:
                hist["span"][r] = (at, at + m)
            at += m
        if graph and new == [1, 1, 1]:
            if not decode:
                st = dict(rows=i32(which), new=i32(new), qkv=qkv.clone(),
                          q_out=torch.empty((3, hq, d), dtype=torch.bfloat16, device="cuda"),
                          out=torch.empty((3, hq, d), dtype=torch.bfloat16, device="cuda"))
                torch.cuda.synchronize()
                cg = torch.cuda.CUDAGraph()
                with torch.cuda.graph(cg):
                    p.plan(st["new"], 3, rows=st["rows"])
                    run(st["qkv"], st["q_out"], st["out"])
                decode.update(st, g=cg)
            decode["rows"].copy_(i32(which))
            decode["qkv"].copy_(qkv)
            decode["g"].replay()
            out = decode["out"].clone()
        else:
            p.plan(i32(new), n, rows=i32(which), max_new=max(new))
            q_out = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
            out = torch.empty_like(q_out)
            run(qkv, q_out, out)
        want = plain_step(hist, qkv, None, hq, hkv, d, pairing, wq, wk, cache, sk, sv)
        torch.cuda.synchronize()
        for r, (a, b) in hist["span"].items():
            # codes and bf16 values may fall on the other side of a rounding
            # border in fp32: a relative norm, not a value's bound
            o = out[a:b].double()
            assert float((o - want[r]).norm() / want[r].norm()) < 2.0 ** -7, (step, r)
            hist["len"][r] += b - a
        assert p.lengths.tolist() == hist["len"]
    assert errors(p) == 0


def test_calls_on_a_stream_of_their_own():
    p, s = filled(4, 2, 64, 32, [400, 3], [1, 1], "bf16", seed=9)
    want, tol = attention_64(p, s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(s["q"])
    p.attention(0, s["q"], out=out, stream=st)
    st.synchronize()
    close(out, want, tol)


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("new", [[1, 1], [200, 3]])
def test_a_wait_that_gives_up(new, cache):
    """... is reported, and the next plan's calls are right again."""
    p, s = filled(4, 2, 128, 32, [4000, 3], new, cache, seed=9)
    want, tol = attention_64(p, s)
    p.set_wait(2_000_000, stall=True)
    out = p.attention(0, s["q"])
    torch.cuda.synchronize()
    assert errors(p) == kv.PAGES_ERR_TIMEOUT
    p.set_wait()
    p.plan(i32(new), sum(new), max_new=max(new))
    p.attention(0, s["q"], out=out)
    close(out, want, tol)


# ---------------------------------------------------------------- refusals
def test_refusals_of_the_binding():
    p, s = filled(4, 2, 64, 16, [20], [4], "bf16", seed=1)
    q = s["q"]
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(causal=False, window=3), dict(window=-1), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan)):
        with pytest.raises(kv.KvRingError):
            p.attention(0, q, **bad)
    for bad in (q.float(), q[:, :3], q[..., :32], q.cpu(), q.transpose(0, 1).contiguous().transpose(0, 1), q[0]):
        with pytest.raises(ValueError):
            p.attention(0, bad)
    with pytest.raises(kv.KvRingError):
        p.attention(1, q)
    with pytest.raises(kv.KvRingError):
        p.attention(0, q, out=q)
    with pytest.raises(kv.KvRingError):   # 4 tokens of 9, off by 8 bytes
        p.attention(0, torch.zeros(4 * 256 + 8, dtype=torch.bfloat16, device="cuda")[4:4 + 1024].view(4, 4, 64))
    with pytest.raises(kv.KvRingError):
        p.attention(0, torch.zeros((5, 4, 64), dtype=torch.bfloat16, device="cuda"))   # beyond max_tokens
    with pytest.raises(kv.KvRingError):
        p.write(0, q, k, k, q_out=q)
    with pytest.raises(kv.KvRingError):
        p.write(0, q, k, k, eps=-1.0)
    with pytest.raises(ValueError):
        p.write(0, q, k[:3], k)
    with pytest.raises(ValueError):
        p.write(0, q, k, k, q_norm=torch.ones(64, device="cuda"))
    with pytest.raises(kv.KvRingError):
        p.set_scales(0, torch.ones(2, device="cuda"), torch.ones(2, device="cuda"))   # a bf16 cache has none
    with pytest.raises(ValueError):
        p.plan(torch.ones(1, dtype=torch.int64, device="cuda"), 4)
    with pytest.raises(ValueError):
        p.plan(i32([1]), 4, rows=i32([0, 1]))
    for args in ((i32([1]), 0), (i32([1]), 5), (i32([1, 1]), 2)):
        with pytest.raises(kv.KvRingError):
            p.plan(*args)
    with pytest.raises(kv.KvRingError):
        p.plan(i32([1]), 4, max_new=0)
    with pytest.raises(kv.KvRingError):
        p.plan(i32([1]), 2 ** 32 + 4)   # does not wrap to 4
    with pytest.raises(kv.KvRingError):
        p.attention(2 ** 32, q)
    with pytest.raises(ValueError):
        p.restore(i32([1, 2]), p.tables, i32([0]))
    assert errors(p) == 0


# ------------------------------------------------------------ other streams
def busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(40_000_000)   # some 20 ms


def test_results_made_on_another_stream():
    """Neither earlier work of the current stream, in memory that was freed
    there, nor later work of it, in the result's once it is dropped, meets a
    call on a stream of its own."""
    p, s = filled(4, 2, 64, 32, [400, 300], [1, 200], "bf16", seed=9)
    k = torch.ones((201, 2, 64), dtype=torch.bfloat16, device="cuda")
    want, tol = attention_64(p, s)
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    before_k, before_v = p.k_cache(0).clone(), p.v_cache(0).clone()
    q_want = p.write(0, s["q"], k, k)
    p.k_cache(0).copy_(before_k)
    p.v_cache(0).copy_(before_v)
    torch.cuda.synchronize()
    for call, result in ((lambda: p.attention(0, s["q"], stream=side), None),
                         (lambda: p.write(0, s["q"], k, k, stream=side), q_want)):
        olds = [torch.empty_like(s["q"]) for _ in range(4)]
        busy(here)
        for x in olds:
            x.fill_(7.0)      # still to come when the call below runs
        del olds, x
        out = call()
        torch.cuda.synchronize()
        close(out, want, tol) if result is None else close(out, result.double(), 0.0)
        busy(side)
        out = call()
        del out
        later = [torch.full_like(s["q"], 7.0) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(bool((x == 7.0).all()) for x in later)


def test_a_cache_made_on_another_stream():
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    make = lambda **kw: kv.KvPages(2, 1, 64, 16, 40, 6, 200, 64, **kw)  # noqa: E731
    old = make().buf
    n = old.numel()
    torch.cuda.synchronize()
    busy(here)
    old.fill_(7)
    del old
    p = make(stream=side)
    torch.cuda.synchronize()
    assert p.nbytes == n and p.free_pages.tolist() == list(range(39, -1, -1))
    assert p.lengths.tolist() == [0] * 6 and errors(p) == 0


# -------------------------------------------------------- ranges of numbers
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_far_below_the_largest_over_e4m3(d, new):
    """Values that only tokens of weight 2^-23.5 of the largest have, beside
    it in the same tile: their probabilities keep their bits in f16."""
    p, s = filled(2, 1, d, 16, [300], [new], "e4m3", seed=2, garbage=False)
    k, v, q = torch.zeros_like(p.k_cache(0), dtype=torch.float32), torch.zeros_like(p.v_cache(0), dtype=torch.float32), s["q"]
    ids = p.tables[0].long()
    k[ids[200 // 16], 0, 200 % 16, 0] = 448.0
    for j in range(192, 208):
        v[ids[j // 16], 0, j % 16] = 0.0 if j == 200 else 448.0
    p.k_cache(0).copy_(k.to(torch.float8_e4m3fn))
    p.v_cache(0).copy_(v.to(torch.float8_e4m3fn))
    s["sk"].fill_(23.5 * math.log(2.0) * math.sqrt(d) / 448.0)
    s["sv"].fill_(1.0)
    p.set_scales(0, s["sk"], s["sv"])
    q.zero_()
    q[..., 0] = 1.0
    want, _ = attention_64(p, s)
    # a probability of 2^-16.5 behind the shift of 2^7 in steps of 2^-24, the
    # result to bf16, and 2^-12 for fp32 scores of 23.5 and their exponentials
    close(p.attention(0, q), want, (2.0 ** -8.5 + 2.0 ** -8 + 2.0 ** -12) * want)
    assert errors(p) == 0


@pytest.mark.parametrize("rise", [0.0, 7.9])
@pytest.mark.parametrize("d,total,new", [(128, 300, 1), (128, 6000, 60), (64, 5000, 3), (64, 700, 300), (128, 20000, 1)])
def test_values_at_the_end_of_bf16(d, total, new, rise):
    """Values up to 3.3e38 under scores that rise by less than what raises a
    running maximum: sums over thousands of tokens that stay finite."""
    p, s = filled(2, 2, d, 32, [total], [new], "bf16", seed=15, garbage=False)
    g = torch.Generator(device="cuda").manual_seed(1)
    p.v_cache(0).copy_((1.0e38 + 2.3e38 * torch.rand(p.v_cache(0).shape, generator=g, device="cuda")).to(torch.bfloat16))
    c, j = p.k_cache(0), torch.arange(total, device="cuda")
    x = c.float()
    x[..., 0] = 0.0
    x[p.tables[0, j // 32].long(), :, j % 32, 0] = (j * (1.0 / total))[:, None].expand(total, 2)
    c.copy_(x.to(torch.bfloat16))
    q = 0.05 * s["q"].float()
    q[..., 0] = rise * math.log(2.0) * math.sqrt(d)
    q = q.to(torch.bfloat16)
    want, tol = attention_64(p, s, q=q)
    out = p.attention(0, q)
    assert bool(torch.isfinite(out).all())
    close(out, want, tol)
    # and small ones keep theirs
    p.v_cache(0).mul_(2.0 ** -190)
    want, tol = attention_64(p, s, q=q)
    close(p.attention(0, q).double() * 2.0 ** 100, want * 2.0 ** 100, (tol - 1e-30) * 2.0 ** 100)
    assert errors(p) == 0


@pytest.mark.parametrize("new", [1, 3, 50])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_of_the_last_exponent_over_e4m3(d, new):
    """Finite bf16 queries from 2^127 on, under scales that leave moderate scores."""
    p, s = filled(4, 2, d, 32, [300], [new], "e4m3", seed=16)
    p.k_cache(0).copy_((p.k_cache(0).float() * 0.01).to(torch.float8_e4m3fn))
    s["sk"].fill_(2.0 ** -126)
    p.set_scales(0, s["sk"], s["sv"])
    q = s["q"].float()
    q = ((1.0 + 0.9 * (q - q.floor())) * 2.0 ** 126 * 2.0 * torch.where(q > 0, 1.0, -1.0)).to(torch.bfloat16)
    q[0, 0] = s["q"][0, 0]        # a row of common size among them
    assert bool(torch.isfinite(q).all())
    want, tol = attention_64(p, s, q=q)
    close(p.attention(0, q), want, tol)
    assert errors(p) == 0


# ------------------------------------------------------------------ release
def test_release_puts_back_no_page_that_the_pool_does_not_have():
    p = pool(16, 100, 4, 1600, 64)
    ids = torch.full((4, 100), -1, dtype=torch.int32, device="cuda")
    ids[0, :3] = torch.tensor([5, 99, 100], dtype=torch.int32)
    ids[1, :70] = torch.arange(20, 90, dtype=torch.int32)
    ids[1, 33], ids[1, 64], ids[1, 0] = -7, 2 ** 31 - 1, -1
    ids[2, :1] = 6
    p.restore(i32([48, 70 * 16 - 3, 1, 0]), ids, i32([1, 2]))
    p.release(i32([3, 2]))
    assert errors(p) == 0 and p.free_pages[:3].tolist() == [1, 2, 6]
    p.release(i32([1, 0]))
    want = [1, 2, 6] + [i for i in range(20, 90) if i not in (20, 53, 84)] + [5, 99]
    assert errors(p) == kv.PAGES_ERR_TABLE
    assert p.lengths.tolist() == [0] * 4 and p.state[kv.PAGES_STATE["free"]].item() == len(want)
    assert p.free_pages[:len(want)].tolist() == want
    assert bool((p.tables == -1).all())
    # an id that a plan took from the free list and that is no page goes out of circulation too
    p.state[kv.PAGES_STATE["error"]] = 0
    p.restore(i32([0] * 4), ids.fill_(-1), i32([3, 4, 777]))
    p.plan(i32([40]), 40)
    assert errors(p) == kv.PAGES_ERR_TABLE
    p.commit()
    p.release(i32([0]))
    assert p.state[kv.PAGES_STATE["free"]].item() == 2 and sorted(p.free_pages[:2].tolist()) == [3, 4]


# ------------------------------------------------------- beside the ring
def test_a_plans_positions_as_a_rings_query_positions():
    """The ring's attention reads its query positions before it waits, unless
    a kernel in flight writes them."""
    H, d, n = 4, 64, 50
    ring = kv.KvRing(H, d, 300, n, 2000)
    p = pool(16, 400, 3, 1900, n, cache_dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = [torch.randn((n, H, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    ring.calibrate(x[1], x[2])
    for _ in range(6):
        ring.write(x[1], x[2])
    starts = [[0, 700, 31], [1500, 2, 900], [64, 64, 1800]]
    new = [i32([20, 0, 30]), i32([1, 48, 1]), i32([7, 7, 7])]
    tables = torch.arange(3 * p.W, dtype=torch.int32, device="cuda").view(3, p.W) % 400
    want = []
    for lens, k in zip(starts, new):
        p.restore(i32(lens), tables, i32(list(range(200))))
        pos = p.plan(k, n).positions.clone()
        torch.cuda.synchronize()
        want.append(ring.attention(x[0], qpos=pos))
    assert errors(p) == 0 and not torch.equal(want[0], want[1])
    lens = [i32(s) for s in starts]
    free = i32(list(range(200)))
    torch.cuda.synchronize()
    for i in range(60):
        p.restore(lens[i % 3], tables, free)
        step = p.plan(new[i % 3], n)
        before = kv.late_reads()
        out = ring.attention(x[0], qpos=step.positions)
        assert kv.late_reads() == before + 1
        assert torch.equal(out, want[i % 3]), i
    # a write of the ring in between lets the plan's kernel stay in flight
    step = p.plan(new[0], n)
    ring.write(x[1], x[2])
    before = kv.late_reads()
    ring.attention(x[0], qpos=step.positions)
    assert kv.late_reads() == before + 1


def test_arguments_in_the_caches_own_buffer():
    p, s = filled(4, 1, 64, 16, [20, 40], [4, 4], "bf16", seed=1)
    p.commit()
    q = s["q"]
    k = torch.zeros((8, 1, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    state = [t.clone() for t in (p.lengths, p.tables, p.free_pages)]
    n = p.state[kv.PAGES_STATE["free"]].item()
    p.restore(p.lengths, p.tables, p.free_pages[:n])     # as they are
    step = p.plan(i32([1, 1]), 8)
    assert step.lengths.tolist() == [21, 41] and errors(p) == 0
    p.restore(state[0], state[1], p.free_pages[:n])
    assert all(torch.equal(a, b) for a, b in zip(state, (p.lengths, p.tables, p.free_pages)))
    other = torch.zeros_like(p.tables)
    with pytest.raises(kv.KvRingError):
        p.restore(p.lengths, p.tables, p.free_pages[1:n])
    with pytest.raises(kv.KvRingError):
        p.restore(p._klen, other, i32([0]))
    with pytest.raises(kv.KvRingError):
        p.plan(p._klen, 8)
    with pytest.raises(kv.KvRingError):
        p.plan(i32([1, 1]), 8, rows=p._slots[:2])
    own = p.k_cache(0).view(-1)[:8 * 4 * 64].view(8, 4, 64)
    with pytest.raises(kv.KvRingError):
        p.attention(0, q, out=own)
    with pytest.raises(kv.KvRingError):
        p.write(0, q, k, k, q_out=own)
    out = torch.zeros(8 * 4 * 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(kv.KvRingError):
        p.write(0, q, k, k, k_norm=out[64:128], q_out=out.view(8, 4, 64))
    p.write(0, q, k, k, k_norm=w, q_out=out.view(8, 4, 64))
    assert errors(p) == 0 and all(torch.equal(a, b) for a, b in zip(state[:1], (p.lengths,)))
