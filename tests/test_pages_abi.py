"""Host-only checks of the paged cache's C ABI: layout, configs and refusals
that need no GPU."""
import ctypes

import pytest

import ring_kv_cache_gb300 as kv


def config(**kw):
    c = kv.make_pages_config(32, 8, 128, 64, 1000, 16, 20, 512, layers=3)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_layout_holds_every_part_in_order():
    lay = kv.kvring_pages_get_layout(config())
    cache = 3 * 1000 * 8 * 64 * 128
    assert (lay.k_cache, lay.v_cache, lay.scales) == (0, cache, 2 * cache)
    names = [f for f, _ in lay._fields_]
    offs = [getattr(lay, f) for f in names]
    assert offs == sorted(offs) and all(o % 256 == 0 for o in offs)
    assert lay.free_pages - lay.tables >= 16 * 20 * 4 and lay.slots - lay.positions >= 512 * 4
    assert kv.kvring_pages_get_layout(config(cache_dtype=kv.CACHE_BF16)).v_cache == 2 * cache


@pytest.mark.parametrize("field,value", [
    ("num_q_heads", 0), ("num_q_heads", 31), ("num_kv_heads", 0), ("num_q_heads", 8 * 65), ("head_dim", 96),
    ("num_layers", 0), ("page_size", 8), ("page_size", 48), ("page_size", 512), ("num_pages", 0),
    ("num_pages", 1 << 22), ("max_requests", 0), ("max_requests", 4097), ("max_pages_per_request", 0),
    ("max_pages_per_request", (1 << 18) + 1), ("max_tokens", 0), ("max_tokens", (1 << 20) + 1), ("cache_dtype", 2),
    ("rope_pairing", 2), ("reserved", 1), ("rope_base", 0.0), ("rope_base", float("nan"))])
def test_bad_configs_are_rejected(field, value):
    with pytest.raises(kv.KvRingError):
        kv.kvring_pages_get_layout(config(**{field: value}))


def test_null_arguments_are_refused_without_a_gpu():
    L, c, out = kv.lib(), config(), ctypes.c_void_p()
    assert L.kvring_pages_get_layout(ctypes.byref(c), None) == 1
    assert L.kvring_pages_create(ctypes.byref(c), None, 1 << 40, None, ctypes.byref(out)) == 1
    assert L.kvring_pages_create(ctypes.byref(c), 0x1001, 1 << 40, None, ctypes.byref(out)) == 1
    assert L.kvring_pages_create(ctypes.byref(c), 0x1000, 1 << 10, None, ctypes.byref(out)) == 3
    assert L.kvring_pages_create(None, 0x1000, 1 << 40, None, ctypes.byref(out)) == 1
    assert L.kvring_pages_restore(None, None, None, None, 0, None) == 1
    assert L.kvring_pages_set_scales(None, 0, None, None, None) == 1
    assert L.kvring_pages_plan(None, None, None, 1, 1, 1, None) == 1
    assert L.kvring_pages_commit(None, None) == 1
    assert L.kvring_pages_release(None, None, 1, None) == 1
    assert L.kvring_pages_write(None, 0, None, None, None, 0, 0, 0, None, None, 0.0, None, 1, None) == 1
    assert L.kvring_pages_attention(None, 0, None, 0, None, 1, 1, 0, 0.0, None) == 1
    assert L.kvring_pages_debug_set_wait(None, 1000, 0) == 1
    assert L.kvring_pages_destroy(None) == 0


@pytest.mark.parametrize("at", range(9))
def test_config_integers_do_not_wrap(at):
    args = [32, 8, 128, 64, 1000, 16, 20, 512, 3]
    good = kv.kvring_pages_get_layout(kv.make_pages_config(*args))
    assert good.total > 0
    for by in (2 ** 32, -2 ** 32, 2 ** 33):
        bad = list(args)
        bad[at] += by
        with pytest.raises(kv.KvRingError):
            kv.kvring_pages_get_layout(kv.make_pages_config(*bad))
