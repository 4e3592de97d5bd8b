"""residual_norm on the GPU: as many rows as the kernels for throughput take."""
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
