"""Host-only checks of the paged cache's block scales and 3-D positions: layout
and configs, no GPU."""
import ctypes

import pytest

import ring_kv_cache_gb300 as kv


def config(**kw):
    c = kv.make_pages_config(32, 8, 128, 64, 1000, 16, 20, 512, layers=3)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_block_scales_have_a_byte_for_sixteen_tokens():
    plain, blocks = kv.kvring_pages_get_layout(config()), kv.kvring_pages_get_layout(config(scale_block=16))
    n = 3 * 1000 * 8 * 4
    assert plain.k_block_scales == plain.v_block_scales
    assert blocks.v_block_scales - blocks.k_block_scales == (n + 255) // 256 * 256
    assert blocks.total - plain.total == 2 * ((n + 255) // 256 * 256)
    for f in ("k_cache", "v_cache", "scales", "slots"):
        assert getattr(plain, f) == getattr(blocks, f)


def test_the_table_has_a_row_per_coordinate():
    row = 128 * 4
    at = lambda **kw: kv.kvring_pages_get_layout(config(**kw)).total  # noqa: E731
    base = at()
    assert at(rope_pairs_t=16, rope_pairs_y=24) == base
    assert at(rope_pairs_t=16, rope_pairs_y=24, max_position=100) == base - (20 * 64 - 100) * row
    assert at(rope_pairs_t=16, max_position=1 << 20) == base + ((1 << 20) - 20 * 64) * row


@pytest.mark.parametrize("fields", [
    dict(scale_block=8), dict(scale_block=32), dict(scale_block=-16), dict(scale_block=16, cache_dtype=kv.CACHE_BF16),
    dict(rope_pairs_y=4), dict(rope_frequencies=1), dict(max_position=10), dict(rope_pairs_t=-1), dict(rope_pairs_t=65),
    dict(rope_pairs_t=40, rope_pairs_y=25), dict(rope_pairs_t=8, rope_pairs_y=-1), dict(rope_pairs_t=8, rope_frequencies=2),
    dict(rope_pairs_t=8, max_position=-1), dict(rope_pairs_t=8, max_position=(1 << 24) + 1), dict(reserved2=1),
    dict(rope_pairs_t=1, rope_pairs_y=2 ** 31 - 1)])
def test_bad_configs_are_refused(fields):
    with pytest.raises(kv.KvRingError):
        kv.kvring_pages_get_layout(config(**fields))


@pytest.mark.parametrize("fields", [
    dict(scale_block=16), dict(rope_pairs_t=64), dict(rope_pairs_t=1, rope_pairs_y=63), dict(rope_pairs_t=22, rope_pairs_y=21,
                                                                                       rope_frequencies=1, max_position=1)])
def test_good_configs_are_taken(fields):
    assert kv.kvring_pages_get_layout(config(**fields)).total > 0


def test_integers_do_not_wrap():
    for kw in (dict(scale_block=2 ** 32 + 16), dict(rope3d=(2 ** 32 + 8, 8)), dict(rope3d=(8, 2 ** 32 + 8)),
               dict(rope3d=(8, 8), max_position=2 ** 32 + 5), dict(rope3d=(8, 8), rope_frequencies=2 ** 32)):
        with pytest.raises(kv.KvRingError):
            kv.kvring_pages_get_layout(kv.make_pages_config(32, 8, 128, 64, 1000, 16, 20, 512, **kw))


def test_null_arguments_are_refused():
    assert kv.lib().kvring_pages_write_3d(None, 0, None, None, None, 0, 0, 0, None, None, 0.0, None, None, 1, None) == 1
    assert ctypes.sizeof(kv.KvringPagesConfig) == 48 + 8 + 24
