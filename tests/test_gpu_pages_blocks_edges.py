"""Block scales on the GPU at the ends of their range: the largest queries over
the largest keys, and steps whose tokens were all skipped."""
import pytest
import torch

import ring_kv_cache_gb300 as kv
from _blockscheck import B, HIGH, LOW, cache_of
from _pagescheck import close, errors
from test_gpu_pages_blocks import inputs, places, run

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def values(p, b, n):
    """float64 [n, d]: the values of head 0 of request b's tokens."""
    at = torch.arange(n, device="cuda")
    ids = p.tables[b, at // p.P].long()
    codes = p.v_cache(0).view(torch.uint8)[ids, 0, at % p.P].view(torch.float8_e4m3fn).double()
    e = p.v_scales(0).view(torch.uint8)[ids, 0, at % p.P // B].double()
    return codes * torch.exp2(e - 127)[:, None]


@pytest.mark.parametrize("exponent", [LOW, 127, HIGH - 9, HIGH])
@pytest.mark.parametrize("size", [2.0 ** 60, 2.0 ** 90, 1.5 * 2.0 ** 127])
@pytest.mark.parametrize("d,new", [(64, 1), (128, 1), (64, 90), (128, 90)])
def test_large_queries_over_large_keys(d, new, size, exponent):
    """Codes of 16 to 448 of either sign: every row is one-hot on its largest score, finite or not in 32 bits.

    The largest code and the next are 192 apart: 2^7 2^-40 2^60 / 2^3 = 2^24 in log2 units at
    least, so nothing else weighs; a single value's way through f16 (2^-11), the division
    (2^-22) and bf16 (2^-8) is left."""
    total = 200
    p, s = cache_of(2, 1, d, 32, [total], [new], seed=31)
    p.k_scales(0).view(torch.uint8).fill_(exponent)
    c = p.k_cache(0)
    x = torch.zeros(c.shape, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(32)
    code = torch.randint(1, 17, (total,), generator=g, device="cuda") * 16.0       # 16 .. 256
    code[::2] *= -1
    code[33], code[118] = 448.0, -448.0
    at = torch.arange(total, device="cuda")
    x[p.tables[0, at // 32].long(), 0, at % 32, 3] = code.to(torch.float8_e4m3fn).float()
    c.copy_(x.to(c.dtype))
    q = torch.zeros_like(s["q"])
    q[..., 3] = size
    q[1::2, :, 3] *= -1
    q[:, 1] *= -1
    out = p.attention(0, q, causal=False).double()
    v = values(p, 0, total)
    for t in range(new):
        for h in range(2):
            want = v[33] if (t + h) % 2 == 0 else v[118]
            close(out[t, h], want, (2.0 ** -8 + 2.0 ** -10) * want.abs(), (t, h))
    assert errors(p) == 0


@pytest.mark.parametrize("d,new", [(64, 1), (128, 1), (64, 90), (128, 90)])
def test_large_queries_keep_blocks_in_order(d, new):
    """Two blocks whose scales differ: the larger score is of the larger scale, whichever code it has."""
    total = 96
    p, s = cache_of(2, 1, d, 32, [total], [new], seed=33)
    ks = p.k_scales(0).view(torch.uint8)
    ks.fill_(HIGH - 4)
    ks[int(p.tables[0, 1]), :, 1] = HIGH          # tokens 48 .. 63
    c = p.k_cache(0)
    x = torch.zeros(c.shape, device="cuda")
    at = torch.arange(total, device="cuda")
    x[p.tables[0, at // 32].long(), 0, at % 32, 5] = 416.0
    x[int(p.tables[0, 1]), 0, 16:32, 5] = 20.0
    x[int(p.tables[0, 1]), 0, 23, 5] = 32.0       # 32 x 2^4 > 416
    c.copy_(x.to(c.dtype))
    q = torch.zeros_like(s["q"])
    q[..., 5] = 2.0 ** 120
    out = p.attention(0, q, causal=False).double()
    want = values(p, 0, total)[48 + 7]
    close(out, want.expand_as(out), (2.0 ** -8 + 2.0 ** -10) * want.abs().expand_as(out))


SKIPS = [([17], [1], [0]), ([32], [16], list(range(16))), ([48], [48], list(range(16, 32))),
         ([40, 16, 5], [8, 16, 5], list(range(16)) + [24, 25]), ([33, 34, 35], [1, 2, 3], [0, 1, 2, 3, 4, 5]), ([21], [2], [0, 1])]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("total,new,bad", SKIPS, ids=[str(i) for i in range(len(SKIPS))])
def test_blocks_whose_tokens_were_all_skipped_stay_as_they_were(total, new, bad, d):
    """Codes and scales both, in a layer that is written again under the same plan too."""
    n = sum(new)
    p, s = cache_of(4, 2, d, 16, total, new, seed=34, rope3d=(8, 12), max_position=100)
    q, k, v, wq, wk = inputs(p, n, 35)
    xyz = places(n, 36, 100)
    good = xyz.clone()
    xyz[bad, 1] = 100
    run(p, s, q, k, v, wq, wk, "adjacent", (8, 12), "section", xyz, skip=bad)
    assert errors(p) == kv.PAGES_ERR_POSITION
    p.state[kv.PAGES_STATE["error"]] = 0
    run(p, s, q, k, v, wq, wk, "adjacent", (8, 12), "section", good)
    assert errors(p) == 0
    run(p, s, q, k, v, wq, wk, "adjacent", (8, 12), "section", xyz, skip=bad)
