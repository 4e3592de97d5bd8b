"""Attention over the paged cache with so many units that every CTA has
several whole ones: both row groups in use, last units that end inside a
group, units cut by range borders, and the same bits from call to call."""
import random

import pytest
import torch

from _pagescheck import attention_64, close, errors, filled

pytestmark = pytest.mark.gpu

SMS = 160   # CTAs of an attention launch, at most


def lengths(requests, tokens, heads_kv, per_unit, seed):
    """New tokens and totals of `requests` requests of up to `tokens` tokens,
    all of more than 16 query rows, with at least three units per CTA."""
    r = random.Random(seed)
    new = [r.randint(max(17, 2 * tokens // 3), tokens) for _ in range(requests - 1)] + [tokens]
    units = sum(-(-n // per_unit) for n in new) * heads_kv
    assert units >= 3 * SMS, units
    assert any(n % per_unit % (per_unit // 2) for n in new)   # a last unit ends inside a group
    return [n + r.choice([0, 1, 127, r.randint(0, 400)]) for n in new], new


def same_bits(p, s, out, calls, **kw):
    for i in range(calls):
        again = p.attention(0, s["q"], **kw)
        differ = (again != out).any(-1).nonzero().tolist()
        assert not differ, ("call", i, differ[:8], len(differ))


# (query heads, key/value heads, requests, most new tokens): Hq / Hkv of 1, 3, 4, 5, 7 and 8
UNITS = [(40, 40, 10, 400), (60, 60, 1, 2200), (36, 12, 9, 500), (64, 16, 3, 900), (40, 8, 8, 500), (56, 8, 7, 400),
         (64, 8, 4, 700), (32, 8, 10, 600)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,cache", [(128, "e4m3"), (64, "e4m3"), (128, "bf16"), (64, "bf16")])
@pytest.mark.parametrize("case", range(len(UNITS)))
def test_many_whole_units_per_cta(case, d, cache, causal):
    hq, hkv, requests, tokens = UNITS[case]
    seed = 100 * case + d + causal
    total, new = lengths(requests, tokens, hkv, 2 * (128 // (hq // hkv)), seed)
    page = random.Random(seed).choice([16, 32, 64, 128, 256])
    p, s = filled(hq, hkv, d, page, total, new, cache, seed=seed)
    out = torch.full_like(s["q"], 9.0)
    p.attention(0, s["q"], out=out, causal=causal)
    want, tol = attention_64(p, s, causal=causal)
    close(out, want, tol)
    same_bits(p, s, out, 20, causal=causal)
    assert errors(p) == 0


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,page,requests,most,new", [
    (32, 8, 128, 64, 60, 4000, 1), (10, 10, 128, 16, 6, 12000, 4), (16, 2, 64, 32, 50, 3000, 2), (7, 1, 64, 16, 128, 2500, 2),
    (8, 8, 64, 256, 30, 5000, 16)])
def test_few_rows_over_many_tiles(hq, hkv, d, page, requests, most, new, cache):
    """Hundreds of tiles per CTA, so that its warps have the room to drift apart."""
    r = random.Random(requests)
    total = [r.randint(most // 8, most) for _ in range(requests)]
    p, s = filled(hq, hkv, d, page, total, [new] * requests, cache, seed=requests)
    out = p.attention(0, s["q"])
    want, tol = attention_64(p, s)
    close(out, want, tol)
    same_bits(p, s, out, 50)
    assert errors(p) == 0


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("d,window", [(64, 0), (64, 60), (128, 60)])
@pytest.mark.parametrize("hq,hkv,requests", [(8, 8, 120), (12, 4, 150), (16, 2, 200)])
def test_units_of_one_tile(hq, hkv, requests, d, window, cache):
    """A unit's end and the next one's only tile follow at once."""
    r = random.Random(requests)
    new = [r.randint(17, 40) for _ in range(requests)]
    total = [n + r.randint(0, 80) for n in new]
    p, s = filled(hq, hkv, d, 16, total, new, cache, seed=d)
    out = p.attention(0, s["q"], window=window)
    want, tol = attention_64(p, s, window=window)
    close(out, want, tol)
    same_bits(p, s, out, 50, window=window)
    assert errors(p) == 0


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,page,singles,chunks", [
    (32, 8, 128, 64, 100, [900, 70]), (10, 10, 128, 16, 16, [757]), (20, 4, 64, 32, 128, [600, 33]), (7, 1, 64, 128, 60, [1500, 1])])
def test_single_tokens_and_chunks_in_one_step(hq, hkv, d, page, singles, chunks, cache):
    """Both kernels in one call, over a serving step's batch."""
    r = random.Random(singles)
    new = [1] * singles + chunks
    r.shuffle(new)
    total = [n + r.randint(0, 2500) for n in new]
    p, s = filled(hq, hkv, d, page, total, new, cache, seed=singles, pad=3)
    out = torch.full_like(s["q"], 9.0)
    p.attention(0, s["q"], out=out)
    n = sum(new)
    want, tol = attention_64(p, s)
    close(out[:n], want[:n], tol[:n])
    for i in range(30):
        again = torch.full_like(out, 9.0)
        p.attention(0, s["q"], out=again)
        assert torch.equal(again, out), i   # rows past the plan's among them
    assert errors(p) == 0
