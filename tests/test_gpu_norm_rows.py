"""residual_norm on the GPU: as many rows as the kernels for throughput take, and
tables that another call has just written."""
import pytest
import torch

import ring_kv_cache_gb300 as kv
from test_gpu_norm import BF, F32, check, reference, tensors
from _pagescheck import close

pytestmark = pytest.mark.gpu


# More rows than the latency form takes (rows x width / 8 > 152 x 1024), no
# multiple of four; five and four groups a thread full and not, two full and
# not, a warp and several for a row.
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("width,n", [(64, 20001), (136, 9303), (256, 5001), (512, 2501), (1016, 2001), (1024, 2003), (1272, 2001),
                                     (1280, 2002), (1288, 2001), (1536, 2001), (2048, 2001), (2560, 1001), (3080, 1001),
                                     (4096, 1003), (5120, 1001), (5128, 501), (8192, 301)])
def test_many_rows(width, n, stream):
    for norm, post, mods in (("rms", "layer", F32), ("layer", "rms", BF), ("rms", None, F32)):
        t = tensors(n, width, stream, mods, rows=7, seed=width)
        check(t, post=post, post_weight=post is not None, norm=norm, weight=True, alpha=0.7, idx=t["idx"].sort()[0])


@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("width", [1280, 5120])
def test_many_rows_in_place_and_alone(width, stream):
    n = 1401
    t = tensors(n, width, stream, rows=3, seed=1)
    idx = t["idx"].sort()[0]
    args = dict(gate=t["mod"][:, 0], scale=t["mod"][:, 1], shift=t["mod"][:, 2], mod_rows=idx, norm="layer")
    a = kv.residual_norm(t["h"], t["y"], **args)
    h = t["h"].clone()
    b = kv.residual_norm(h, t["y"], h_out=h, **args)
    assert b[0] is h and torch.equal(a[0], h) and torch.equal(a[1], b[1])
    _, x = kv.residual_norm(t["h"], norm="rms", weight=t["w"])
    _, (want, tol) = reference(t, y=False, norm="rms", weight=True, modulate=False)
    close(x, want, tol)
    got = kv.residual_norm(t["h"], t["y"], gate=t["mod"][:, 0], mod_rows=idx, norm=None)
    (want, tol), _ = reference(t, norm=None, idx=idx)
    close(got[0], want, tol)


@pytest.mark.parametrize("width,n", [(64, 20001), (5120, 1001)])
def test_fp32_tables_in_the_middle_of_a_sector(width, n):
    """The same bits from tables that are aligned to 16 bytes and no more."""
    t = tensors(n, width, BF, rows=7, seed=2)
    idx = t["idx"].sort()[0]
    mod = torch.zeros((7, 3 * width + 8), dtype=F32, device="cuda")[:, 4:4 + 3 * width].view(7, 3, width)
    mod.copy_(t["mod"])
    assert mod.data_ptr() % 32 == 16
    a, b = check(dict(t, mod=mod), idx=idx), check(t, idx=idx)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("mods", [BF, F32])
@pytest.mark.parametrize("width", [64, 1280])
def test_tables_that_the_call_before_wrote(width, mods, captured):
    """Tables are read through L1, and a call starts while the one before it runs: its reads lie
    behind the wait for that one, so a table that every SM has read before is seen as it now is."""
    n, m, turns = 4001, 5, 12
    t = tensors(n, width, BF, mods, rows=m, seed=3)
    idx = t["idx"]
    table = torch.zeros((m, width), dtype=mods, device="cuda")
    grow = tensors(m, width, F32, F32, rows=m, seed=4)
    add = grow["y"]
    out = [torch.empty((n, width), dtype=BF, device="cuda") for _ in range(turns)]

    def chain(wait):
        for i in range(turns):
            kv.residual_norm(t["h"], norm="rms", scale=table, mod_rows=idx, x_out=out[i])   # every SM reads the table
            wait()
            if mods == F32:      # the stream of a few rows is the table: it grows in place
                kv.residual_norm(table, add, norm=None, h_out=table)
            else:                # or their normed sum is, another one each time
                kv.residual_norm(grow["h"], add, gate=table_f32[i], x_out=table, norm="layer")
            wait()

    table_f32 = torch.randn((turns, m, width), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    chain(torch.cuda.synchronize)
    want = [x.clone() for x in out]
    assert not torch.equal(want[1], want[2])
    last = table.clone()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chain(lambda: None)
    for _ in range(20):
        table.zero_()
        for x in out:
            x.fill_(7.0)
        if captured:
            g.replay()
        else:
            chain(lambda: None)
        assert torch.equal(table, last)
        assert all(torch.equal(x, y) for x, y in zip(out, want))
