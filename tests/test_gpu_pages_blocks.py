"""The paged cache's write with 3-D positions and with block scales on the GPU
against plain 64-bit forms."""
import math
import random

import pytest
import torch

import ring_kv_cache_gb300 as kv
from _blockscheck import B, HIGH, LOW, angles_of, cache_of, check_blocks, turned
from _pagescheck import close, errors, i32

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def inputs(p, n, seed, norm=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H = p.Hq + 2 * p.Hkv
    qkv = torch.randn((n, H, p.d), generator=g, device="cuda") * torch.exp2(torch.randint(-6, 7, (n, H, 1), generator=g, device="cuda"))
    q, k, v = qkv.to(BF).split([p.Hq, p.Hkv, p.Hkv], dim=1)
    wq, wk = [(0.5 + torch.rand(p.d, generator=g, device="cuda")).to(BF) if norm else None for _ in "qk"]
    return q, k, v, wq, wk


def places(n, seed, most=300):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, most, (n, 3), generator=g, device="cuda").to(torch.int32)


def run(p, s, q, k, v, wq, wk, pairing, rope3d=None, frequencies="section", xyz=None, skip=()):
    """One write, and every result of it checked."""
    n, t, layer = q.shape[0], min(s["tokens"], q.shape[0]), s["layer"]
    blocks = p.block_scales
    caches = [p.k_cache(layer).clone(), p.v_cache(layer).clone()]
    scales = [x(layer).view(torch.uint8).clone() for x in (p.k_scales, p.v_scales)] if blocks else None
    q_out = torch.full((n, p.Hq, p.d), 7.0, dtype=BF, device="cuda")
    p.write(layer, q, k, v, q_norm=wq, k_norm=wk, q_out=q_out, pos=xyz)
    torch.cuda.synchronize()
    slots = p._slots[:t].clone()
    at = xyz[:t] if rope3d else p._pos[:t]
    ang = angles_of(p.d, at.clamp(0, p.layout.total if not rope3d else 1 << 20), rope3d, frequencies)
    fp = 2.0 ** -19
    there = torch.ones(t, dtype=torch.bool, device="cuda")
    there[list(skip)] = False
    want, m = turned(q[:t], wq, ang, pairing)
    close(q_out[:t][there], want[there], (2.0 ** -8 * want.abs() + fp * m + 1e-30)[there], "q")
    assert bool((q_out[t:] == 7.0).all()) and bool((q_out[:t][~there] == 7.0).all())
    slots[~there] = -1
    for i, (name, x, w) in enumerate((("k", k, wk), ("v", v, None))):
        want, m = turned(x[:t], w, ang if name == "k" else None, pairing)
        if blocks:
            check_blocks(p, s, name, want, m, slots, p._slots[:t], caches[i], scales[i])
            continue
        cache = (p.k_cache, p.v_cache)[i](layer)
        sl = slots[slots >= 0].long()
        want, m = want[slots >= 0], m[slots >= 0]
        raw = cache.view(torch.uint8) if cache.dtype != BF else cache
        got = raw[sl // p.P, :, sl % p.P]
        if cache.dtype == BF:
            close(got, want, (2.0 ** -8 * want.abs() + fp * m) * (name == "k") + 1e-30, name)
        else:
            sc = s["s" + name].double()[:, None]
            want, m = want / sc, m / sc
            close(got.view(cache.dtype).double(), want.clamp(-448, 448), 2.0 ** -4 * want.abs() + 2.0 ** -10 + fp * m, name)
        other = torch.ones((p.num_pages, p.P), dtype=torch.bool, device="cuda")
        other[sl // p.P, sl % p.P] = False
        a, b = [c.view(torch.uint8).view(p.num_pages, p.Hkv, p.P, -1).transpose(1, 2)[other] for c in (cache, caches[i])]
        assert torch.equal(a, b), name


AXES = [((16, 24), "head", 128), ((22, 21), "section", 128), ((1, 0), "section", 128), ((64, 0), "head", 128), ((30, 34), "section", 128),
        ((5, 13), "head", 64), ((8, 12), "section", 64), ((3, 29), "section", 64)]


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("cache", ["bf16", "e4m3", "blocks"])
@pytest.mark.parametrize("rope3d,frequencies,d", AXES, ids=[str(i) for i in range(len(AXES))])
def test_write_by_three_coordinates(rope3d, frequencies, d, cache, pairing):
    for hq, hkv, page, total, new, pad in ((4, 2, 16, [37, 1, 64, 20], [3, 1, 0, 17], 5), (7, 1, 64, [1], [1], 0),
                                           (10, 10, 128, [300, 129], [150, 40], 1)):
        p, s = cache_of(hq, hkv, d, page, total, new, seed=1, layers=2, layer=1, pairing=pairing, pad=pad, cache=cache,
                        rope3d=rope3d, frequencies=frequencies, max_position=301)
        n = sum(new) + pad
        q, k, v, wq, wk = inputs(p, n, 2, norm=hq != 7)
        xyz = places(n, 3)
        xyz[sum(new):] = -5      # padding is not looked at
        run(p, s, q, k, v, wq, wk, pairing, rope3d, frequencies, xyz)
        assert errors(p) == 0


def test_equal_coordinates_turn_as_one_position_does():
    """The frequencies of the whole head: text tokens have the same bits as with 1-D RoPE."""
    a, s = cache_of(4, 2, 128, 32, [200], [60], seed=4, cache="bf16", pairing="halves")
    b, _ = cache_of(4, 2, 128, 32, [200], [60], seed=4, cache="bf16", pairing="halves", rope3d=(16, 24), frequencies="head")
    q, k, v, wq, wk = inputs(a, 60, 5)
    xyz = a._pos[:60, None].expand(60, 3).contiguous()
    one, three = a.write(0, q, k, v, wq, wk), b.write(0, q, k, v, wq, wk, pos=xyz)
    assert torch.equal(one, three) and torch.equal(a.k_cache(0).view(torch.int16), b.k_cache(0).view(torch.int16))


@pytest.mark.parametrize("cache", ["bf16", "blocks"])
@pytest.mark.parametrize("d", [64, 128])
def test_coordinates_that_the_table_does_not_have(cache, d):
    p, s = cache_of(4, 2, d, 16, [70, 40], [50, 3], seed=6, cache=cache, rope3d=(8, 12), max_position=100)
    q, k, v, wq, wk = inputs(p, 53, 7)
    xyz = places(53, 8, 100)
    bad = {3: (0, -1), 20: (1, 100), 21: (2, 2 ** 31 - 1), 36: (0, -2 ** 31), 50: (2, 100)}
    for t, (a, x) in bad.items():
        xyz[t, a] = x
    run(p, s, q, k, v, wq, wk, "adjacent", (8, 12), "section", xyz, skip=list(bad))
    assert errors(p) == kv.PAGES_ERR_POSITION


# -------------------------------------------------------------- block scales
CASES = [
    # hq, hkv, d, page, total, new, pad
    (4, 2, 64, 16, [37, 1, 64, 20], [3, 1, 0, 17], 5),
    (10, 10, 128, 64, [1], [1], 0),
    (7, 1, 128, 128, [300, 129], [150, 1], 1),
    (40, 8, 64, 256, [700], [500], 0),
    (3, 3, 64, 32, [33] * 9, [1] * 9, 3),
    (8, 8, 128, 64, [16, 32, 48, 17, 31, 15], [16, 1, 33, 1, 15, 15], 0),
    (5, 5, 128, 16, [100, 99, 98, 7, 45], [1, 1, 1, 7, 30], 2),
    (2, 1, 64, 64, [50 + i for i in range(40)], [1 + i % 5 for i in range(40)], 0),
]


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_write_into_blocks(case, pairing):
    hq, hkv, d, page, total, new, pad = case
    for norm in (True, False):
        p, s = cache_of(hq, hkv, d, page, total, new, seed=11, layers=2, layer=1, pairing=pairing, pad=pad)
        q, k, v, wq, wk = inputs(p, sum(new) + pad, 12, norm)
        k[sum(new):] = v[sum(new):] = q[sum(new):] = math.nan   # padding has no effect
        run(p, s, q, k, v, wq, wk, pairing)
        run(p, s, q, k, v, wq, wk, pairing)                     # again: the scales are there already
        assert errors(p) == 0


@pytest.mark.parametrize("seed", range(8))
def test_runs_of_any_lengths(seed):
    """Requests of any numbers of new tokens, so that blocks begin and end anywhere in the step."""
    rng = random.Random(seed)
    n = rng.randint(1, 60)
    new = [rng.choice([0, 1, 1, 2, 3, rng.randint(0, 20), rng.randint(10, 70)]) for _ in range(n)]
    new[0] = max(1, new[0])
    total = [x + rng.choice([0, 0, 1, rng.randint(0, 80)]) for x in new]
    total = [max(1, t) for t in total]
    new = [min(a, b) for a, b in zip(new, total)]
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 256])
    p, s = cache_of(3, 3, d, page, total, new, seed=seed + 20)
    q, k, v, wq, wk = inputs(p, sum(new), seed + 30)
    run(p, s, q, k, v, wq, wk, "adjacent")


def test_fewer_tokens_than_planned_and_pages_that_are_none():
    p, s = cache_of(4, 2, 64, 16, [90, 40], [80, 7], seed=13, missing={(0, 2), (0, 3), (1, 2)})
    slots = p._slots[:87].tolist()
    assert slots.count(-1) == 32 + 7 and errors(p) == kv.PAGES_ERR_TABLE
    q, k, v, wq, wk = inputs(p, 87, 14)
    run(p, s, q, k, v, wq, wk, "adjacent")
    for n in (1, 5, 6, 7, 22, 80, 83):
        run(p, s, q[:n].contiguous(), k[:n].contiguous(), v[:n].contiguous(), wq, wk, "adjacent")


def test_a_block_filled_token_by_token():
    """Scales rise while a block fills; every code stays within its rounding steps."""
    p, s = cache_of(2, 2, 64, 32, [1], [1], seed=15, spare=8)
    p.release(i32([0]))
    g = torch.Generator(device="cuda").manual_seed(16)
    n = 32
    x = (torch.randn((n, 2, 64), generator=g, device="cuda") * torch.exp2(torch.arange(n, device="cuda") * 0.4)[:, None, None]).to(BF)
    q = torch.zeros((1, 2, 64), dtype=BF, device="cuda")
    for t in range(n):
        p.plan(i32([1]), 1)
        p.write(0, q, x[t:t + 1], x[t:t + 1])
        p.commit()
    page = int(p.tables[0, 0])
    for blk in range(2):
        sc = p.v_scales(0)[page, :, blk].float()
        part = x[16 * blk:16 * blk + 16].float()
        assert torch.equal(sc.log2().round(), (part.abs().amax((0, 2)) / 448).log2().ceil())
        got = p.v_cache(0)[page, :, 16 * blk:16 * blk + 16].float() * sc[:, None, None]
        # at most one step of E4M3 per value: later moves round only among the subnormals
        tol = 2.0 ** -4 * part.abs().transpose(0, 1) + 16 * 2.0 ** -10 * sc[:, None, None]
        assert bool(((got - part.transpose(0, 1)).abs() <= tol).all())


def test_block_extremes():
    """Zeros, the largest and smallest values, infinities and NaN."""
    p, s = cache_of(2, 2, 64, 16, [16 * 8], [16 * 8], seed=17, spare=0)
    x = torch.ones((128, 6, 64), dtype=BF, device="cuda")
    x[0:16] = 0.0
    x[16:32] = 3e38                       # saturates at 448 * 2^40
    x[32:48] = 1e-30                      # vanishes below 2^-40 * 2^-10
    x[48, :, 5], x[49, :, 6] = math.inf, -math.inf
    x[64, :, 9] = math.nan
    x[80:96] = 448.0                      # exactly the end of a binade's range
    x[96:112] = 450.0
    q, k, v = x.split([2, 2, 2], dim=1)
    p.write(0, q, k, v)
    sl = p._slots[:128].long()
    vc = p.v_cache(0).view(torch.uint8)[sl // 16, :, sl % 16].view(torch.float8_e4m3fn).float()
    e = p.v_scales(0).view(torch.uint8)[sl[::16] // 16, :, 0].int()
    assert e[:, 0].tolist() == [LOW, HIGH, LOW, 119, 119, 127, 128, 119] and torch.equal(e[:, 0], e[:, 1])
    assert bool((vc[0:16] == 0).all()) and bool((vc[16:32] == 448).all()) and bool((vc[32:48] == 0).all())
    assert bool((vc[48, :, 5] == 448).all()) and bool((vc[49, :, 6] == -448).all()) and bool((vc[48, :, 7] == 256).all())
    assert bool(torch.isnan(vc[64, :, 9]).all()) and bool((vc[64, :, 8] == 256).all()) and bool((vc[65] == 256).all())
    assert bool((vc[80:96] == 448).all()) and bool((vc[96:112] == 224).all())


def test_a_captured_write_follows_the_plan():
    """A graph of plan, write and commit: every replay appends where the request then ends."""
    def fresh():
        p, _ = cache_of(4, 2, 128, 16, [30], [5], seed=18, spare=12)
        p.release(i32([0]))
        return p

    a, b = fresh(), fresh()
    q, k, v, wq, wk = inputs(a, 5, 19)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    new = i32([5])
    q_out = torch.empty_like(q)

    def step(p):
        p.plan(new, 5)
        p.write(0, q, k, v, wq, wk, q_out=q_out)
        p.commit()

    step(b)   # (outside the graph first)
    b.release(i32([0]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b)
    for i in range(6):
        k.mul_(1.7)
        step(a)
        want = q_out.clone()
        g.replay()
        assert torch.equal(q_out, want)
    assert a.lengths.tolist() == b.lengths.tolist() == [30]
    for w in range(2):
        pa, pb = int(a.tables[0, w]), int(b.tables[0, w])
        n = min(16, 30 - 16 * w)
        for x in ("k", "v"):
            ca, cb = [getattr(p, x + "_cache")(0).view(torch.uint8)[pg, :, :n] for p, pg in ((a, pa), (b, pb))]
            sa, sb = [getattr(p, x + "_scales")(0).view(torch.uint8)[pg] for p, pg in ((a, pa), (b, pb))]
            assert torch.equal(ca, cb) and torch.equal(sa, sb)


def test_refusals():
    mk = lambda **kw: kv.KvPages(2, 2, 64, 16, 8, 2, 64, 32, **kw)  # noqa: E731
    for kw in (dict(block_scales=True, cache_dtype=BF), dict(rope3d=(0, 4)), dict(rope3d=(33, 0)), dict(rope3d=(8, 25)), dict(rope3d=(8, -1)),
               dict(rope3d=(8,)), dict(rope3d=8), dict(rope3d=(8, None)), dict(rope3d=(8, 8), rope_frequencies="all"), dict(rope_frequencies="head"), dict(max_position=10),
               dict(rope3d=(8, 8), max_position=0), dict(rope3d=(8, 8), max_position=(1 << 24) + 1)):
        with pytest.raises(ValueError):
            mk(**kw)
    plain, blocks, three = mk(), mk(block_scales=True), mk(rope3d=(8, 8), max_position=50)
    with pytest.raises(ValueError):
        plain.k_scales()
    with pytest.raises(ValueError):
        blocks.v_scales(1)
    with pytest.raises(kv.KvRingError) as e:
        blocks.set_scales(0, torch.ones(2, device="cuda"), torch.ones(2, device="cuda"))
    assert e.value.status == 4
    q = torch.ones((4, 2, 64), dtype=BF, device="cuda")
    xyz = torch.zeros((4, 3), dtype=torch.int32, device="cuda")
    for p in (plain, blocks, three):
        p.plan(i32([4]), 4)
    with pytest.raises(ValueError):
        plain.write(0, q, q, q, pos=xyz)
    for bad in (None, xyz[:3], xyz.long(), xyz.t().contiguous().t(), xyz.cpu()):
        with pytest.raises(ValueError):
            three.write(0, q, q, q, pos=bad)
    L = kv.lib()
    args = (q.data_ptr(), q.data_ptr(), q.data_ptr(), 128, 128, 128, None, None, 1e-6)
    out = torch.empty_like(q)
    s = torch.cuda.current_stream().cuda_stream
    assert L.kvring_pages_write(three.handle, 0, *args, out.data_ptr(), 4, s) == 1
    assert L.kvring_pages_write_3d(plain.handle, 0, *args, xyz.data_ptr(), out.data_ptr(), 4, s) == 1
    assert L.kvring_pages_write_3d(three.handle, 0, *args, xyz.data_ptr() + 2, out.data_ptr(), 4, s) == 1
    assert L.kvring_pages_write_3d(three.handle, 0, *args, out.data_ptr() + 64, out.data_ptr(), 4, s) == 1
    assert L.kvring_pages_write_3d(three.handle, 0, *args, three._pos.data_ptr(), out.data_ptr(), 4, s) == 1
    assert L.kvring_pages_write_3d(three.handle, 0, *args, xyz.data_ptr(), out.data_ptr(), 4, s) == 0
