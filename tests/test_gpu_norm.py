"""residual_norm on the GPU against its formula in 64 bits."""
import math

import pytest
import torch

import ring_kv_cache_gb300 as kv
from _pagescheck import close

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def tensors(n, width, stream=BF, mods=F32, rows=1, seed=0, offset=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    h = rand(n, width) * 2 + offset
    h[:, ::37] *= 30.0
    return dict(h=h.to(stream), y=rand(n, width).to(BF), mod=(0.5 * rand(rows, 3, width)).to(mods),
                w=(1 + 0.3 * rand(width)).to(BF), pw=(1 + 0.3 * rand(width)).to(BF),
                idx=torch.randint(0, rows, (n,), generator=g, device="cuda").to(torch.int32))


def standard(z, size, kind, eps):
    """(normed, error in units of 2^-17) of rows that are off by 2^-17 size.

    fp32: a sum of up to 40 terms a thread and 9 halvings is off by 49 x 2^-24
    of the sum of sizes, twice where the mean is taken first; rsqrt 2^-22;
    the factor is off by what the row is, relative to its size."""
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    if kind == "layer":
        z, size = z - mean(z), size + mean(size)
    f = 1 / torch.sqrt(mean(z * z) + eps)
    return z * f, size * f + (z * f).abs() * (1 + torch.sqrt(mean(size * size)) * f)


def reference(t, gate=True, alpha=1.0, post=None, post_weight=False, norm="rms", weight=False, modulate=True, idx=None,
              eps=1e-6, y=True):
    """((h', bound), (x, bound)) in 64 bits."""
    fp, half = 2.0 ** -17, 2.0 ** -8
    h, mod = t["h"].double(), t["mod"].double()
    mod = mod[idx.long()] if idx is not None else mod
    size = h.abs()
    if y:
        u = t["y"].double()
        off = torch.zeros_like(u)
        if post:
            u, off = standard(u, u.abs() * 2.0 ** -6, post, eps)   # (bf16 values are exact: 2^-23 of each)
        if post_weight:
            u, off = u * t["pw"].double(), off * t["pw"].double().abs()
        if gate:
            u, off = u * mod[:, 0], off * mod[:, 0].abs()
        h = h + alpha * u
        size = 2.0 ** -6 * (size + abs(alpha) * u.abs()) + abs(alpha) * off   # in units of 2^-17
    else:
        size = 2.0 ** -6 * size
    tol_h = fp * size + (half * h.abs() if t["h"].dtype == BF else 2.0 ** -24 * h.abs()) + 1e-30
    if not norm:
        return (h, tol_h), None
    x, off = standard(h, size, norm, eps)
    if weight:
        x, off = x * t["w"].double(), off * t["w"].double().abs()
    if modulate:
        x, off = x * (1 + mod[:, 1]) + mod[:, 2], off * (1 + mod[:, 1].abs()) + mod[:, 2].abs()
    return (h, tol_h), (x, half * x.abs() + fp * off + 1e-30)


def check(t, gate=True, alpha=1.0, post=None, post_weight=False, norm="rms", weight=False, modulate=True, idx=None,
          eps=1e-6, **kw):
    mod = t["mod"]
    got = kv.residual_norm(t["h"], t["y"], gate=mod[:, 0] if gate else None, residual_scale=alpha, post_norm=post,
                           post_weight=t["pw"] if post_weight else None, norm=norm, weight=t["w"] if weight else None,
                           scale=mod[:, 1] if modulate else None, shift=mod[:, 2] if modulate else None, mod_rows=idx,
                           eps=eps, **kw)
    (h, th), x = reference(t, gate, alpha, post, post_weight, norm, weight, modulate, idx, eps)
    close(got[0], h, th, "h")
    assert got[0].dtype == t["h"].dtype
    if norm:
        close(got[1], x[0], x[1], "x")
    else:
        assert got[1] is None
    return got


@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("width", [8, 64, 200, 256, 264, 768, 776, 1280, 1288, 2560, 3080, 5120, 5128, 10240, 10248, 16384])
def test_widths(width, stream):
    for n, norm, post in ((1, "rms", "layer"), (7, "layer", "rms"), (130, "rms", None)):
        t = tensors(n, width, stream, seed=n)
        check(t, post=post, post_weight=post is not None, norm=norm, weight=True, alpha=0.7)


@pytest.mark.parametrize("mods", [BF, F32])
@pytest.mark.parametrize("norm", ["rms", "layer", None])
@pytest.mark.parametrize("post", ["rms", "layer", None])
def test_variants(norm, post, mods):
    for gate in (True, False):
        t = tensors(33, 640, F32, mods, rows=5, seed=3)
        tables = gate or norm
        check(t, gate, -1.5, post, False, norm, False, bool(norm), t["idx"] if tables else None, eps=1e-3)
        t = tensors(33, 640, BF, mods, rows=33, seed=4)   # a row each
        check(t, gate, 0.1, post, post is not None, norm, bool(norm), bool(norm))


def test_the_stream_alone():
    t = tensors(12, 136, BF, seed=5)
    h, x = kv.residual_norm(t["h"], norm="layer", weight=t["w"], scale=t["mod"][:, 1], shift=t["mod"][:, 2])
    assert h is t["h"]
    _, (want, tol) = reference(t, y=False, norm="layer", weight=True)
    close(x, want, tol)
    _, x = kv.residual_norm(t["h"], norm="rms")
    _, (want, tol) = reference(t, y=False, norm="rms", modulate=False)
    close(x, want, tol)


def test_strides_in_place_and_what_lies_beside():
    """Slices of packed tensors; in place gives the same bits; nothing beside a result changes."""
    t = tensors(19, 320, F32, rows=4, seed=6)
    wide = lambda x, k: torch.full((x.shape[0] + 2, k), 9.0, dtype=x.dtype, device="cuda")  # noqa: E731
    h, y, ho, xo = wide(t["h"], 648), wide(t["y"], 1000), wide(t["h"], 336), wide(t["y"], 400)
    h[1:20, 8:328], y[1:20, 640:960] = t["h"], t["y"]
    s = dict(t, h=h[1:20, 8:328], y=y[1:20, 640:960])
    a = check(s, idx=t["idx"], post="rms", h_out=ho[1:20, 8:328], x_out=xo[1:20, 40:360])
    assert a[0].data_ptr() == ho[1:20, 8:328].data_ptr()
    for x, lo in ((ho, 8), (xo, 40)):
        m = torch.ones_like(x, dtype=torch.bool)
        m[1:20, lo:lo + 320] = False
        assert bool((x[m] == 9.0).all())
    b = kv.residual_norm(s["h"], s["y"], gate=t["mod"][:, 0], scale=t["mod"][:, 1], shift=t["mod"][:, 2], mod_rows=t["idx"],
                         post_norm="rms", h_out=s["h"])
    assert torch.equal(b[0], a[0]) and torch.equal(b[1], a[1]) and torch.equal(h[1:20, 8:328], a[0])
    assert bool((h[:, :8] == 9.0).all()) and bool((h[0] == 9.0).all())


@pytest.mark.parametrize("width", [64, 1288, 5120])
def test_fp32_rows_that_begin_in_the_middle_of_a_sector(width):
    """16-byte aligned and no more: the rows' 32-byte accesses are two of 16."""
    t = tensors(9, width, F32, rows=3, seed=10)
    beside = lambda x: torch.zeros((x.shape[0], width + 8), dtype=F32, device="cuda")[:, 4:4 + width]  # noqa: E731
    h, ho = beside(t["h"]), beside(t["h"])
    h.copy_(t["h"])
    mod = torch.zeros((3, 3 * width + 8), dtype=F32, device="cuda")[:, 4:4 + 3 * width].view(3, 3, width)
    mod.copy_(t["mod"])
    assert h.data_ptr() % 32 == 16 and mod.data_ptr() % 32 == 16
    a = check(dict(t, h=h, mod=mod), idx=t["idx"], norm="layer", h_out=ho)
    b = check(t, idx=t["idx"], norm="layer")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("width", [64, 1280, 5120])
def test_a_row_that_no_table_has_gets_nan(width):
    t = tensors(10, width, BF, rows=3, seed=7)
    idx = t["idx"].clone()
    idx[2], idx[5], idx[9] = 3, -1, 2 ** 31 - 1
    h, x = kv.residual_norm(t["h"], t["y"], gate=t["mod"][:, 0], scale=t["mod"][:, 1], shift=t["mod"][:, 2], mod_rows=idx)
    bad = torch.zeros(10, dtype=torch.bool, device="cuda")
    bad[[2, 5, 9]] = True
    assert bool(torch.isnan(h[bad]).all()) and bool(torch.isnan(x[bad]).all())
    (hw, th), (xw, tx) = reference(t, idx=t["idx"])
    close(h[~bad], hw[~bad], th[~bad])
    close(x[~bad], xw[~bad], tx[~bad])


@pytest.mark.parametrize("width", [64, 1280, 5120])
def test_rows_without_a_spread_and_values_that_are_not_finite(width):
    t = tensors(8, width, F32, seed=8)
    t["h"][0], t["y"][0] = 0.0, 0.0
    t["h"][1], t["y"][1] = 3.0, 0.0
    h, y = t["h"].clone(), t["y"].clone()
    h[2, 5], h[3, 7], y[4, 1] = math.inf, math.nan, -math.inf
    got_h, x = kv.residual_norm(h, y, norm="layer", scale=t["mod"][:, 1], shift=t["mod"][:, 2])
    (hw, th), (xw, tx) = reference(dict(t, h=h, y=y), gate=False, norm="layer")
    fine = [0, 1, 5, 6, 7]
    close(got_h[fine], hw[fine], th[fine])
    close(x[fine], xw[fine], tx[fine])
    # (rows 0 and 1 are their shift: all values alike)
    close(x[:2], t["mod"][:, 2].double().expand(2, -1), 2.0 ** -8 * t["mod"][:, 2].abs().double() + 3.0 * 2.0 ** -17 * 1e3 *
          (1 + t["mod"][:, 1].abs().double()))
    assert bool(torch.isnan(x[2:5]).all())


def test_the_same_bits_again_on_another_stream_and_in_a_graph():
    t = tensors(300, 1288, BF, rows=6, seed=9)
    args = dict(gate=t["mod"][:, 0], scale=t["mod"][:, 1], shift=t["mod"][:, 2], mod_rows=t["idx"], post_norm="rms", norm="layer")
    a = kv.residual_norm(t["h"], t["y"], **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = kv.residual_norm(t["h"], t["y"], stream=side, **args)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    h, y, xo = t["h"].clone(), t["y"].clone(), torch.empty_like(a[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.residual_norm(h, y, h_out=h, x_out=xo, **args)
        kv.residual_norm(h, y, h_out=h, x_out=xo, **args)
    h.copy_(t["h"])
    g.replay()
    c = kv.residual_norm(a[0], t["y"], **args)
    assert torch.equal(h, c[0]) and torch.equal(xo, c[1])


def test_refusals():
    t = tensors(6, 64, rows=3)
    h, y, mod = t["h"], t["y"], t["mod"]
    ok = dict(gate=mod[:, 0], scale=mod[:, 1], mod_rows=t["idx"])
    kv.residual_norm(h, y, **ok)
    bad = [dict(ok, mod_rows=None), dict(ok, mod_rows=t["idx"].long()), dict(ok, mod_rows=t["idx"][:5]), dict(ok, gate=mod[:, 0].to(BF)),
           dict(ok, shift=mod[:, 2].contiguous()), dict(ok, shift=mod[:2, 2]), dict(ok, norm="batch"), dict(ok, norm=None),
           dict(ok, post_weight=t["pw"]), dict(ok, weight=t["w"][:32]), dict(ok, weight=t["w"].float()), dict(mod_rows=t["idx"]),
           dict(ok, h_out=torch.empty_like(h).float()), dict(ok, x_out=torch.empty_like(h)[:5]), dict(ok, gate=mod[:1, 0].expand(3, 64)),
           dict(ok, gate=mod[:, 0].cpu()), dict(ok, gate=0.5), dict(ok, mod_rows=[0] * 6), dict(ok, weight=1.0), dict(ok, x_out=3)]
    for kw in bad:
        with pytest.raises(ValueError):
            kv.residual_norm(h, y, **kw)
    for kw in (dict(gate=mod[:, 0]), dict(post_norm="rms"), dict(norm=None), dict(h_out=h)):
        with pytest.raises(ValueError):
            kv.residual_norm(h, **kw)
    for a, b in ((h[:, :60], y[:, :60]), (h.half(), y), (h.cpu(), y.cpu()), (h, y[:5]), (h, y.float()), (h[:, ::2], y[:, :32])):
        with pytest.raises(ValueError):
            kv.residual_norm(a, b)
    with pytest.raises(ValueError):
        kv.residual_norm([1.0] * 8, y)
    for kw in (dict(x_out=y), dict(eps=-1.0), dict(residual_scale=math.inf), dict(x_out=h)):
        with pytest.raises(kv.KvRingError):
            kv.residual_norm(h, y, **kw)
    with pytest.raises(kv.KvRingError):
        kv.residual_norm(h[:0], y[:0])
