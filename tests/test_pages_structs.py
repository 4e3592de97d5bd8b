"""Host-only checks of the C structures of the paged cache: those of a program
that knows no block scales and no 3-D positions have the size that they always had,
and nothing behind them is read or written; options come in a structure of their own."""
import ctypes

import pytest

import ring_kv_cache_gb300 as kv

CONFIG = (32, 8, 128, 3, 64, 1000, 16, 20, 512, 0, 0, 0)   # the twelve integers, in the header's order
CONFIG_BYTES, LAYOUT_WORDS, GUARD = 56, 13, 4


def config_of(behind):
    """A config as such a program has it: 56 bytes, and what happens to lie behind them."""
    b = (ctypes.c_uint8 * (CONFIG_BYTES + 64))(*([behind] * (CONFIG_BYTES + 64)))
    ctypes.memmove(b, (ctypes.c_int32 * 12)(*CONFIG), 48)
    ctypes.memmove(ctypes.addressof(b) + 48, (ctypes.c_double * 1)(10000.0), 8)
    return b


def at(f, *args):
    """The C function by its address, without the binding's types."""
    return ctypes.CFUNCTYPE(ctypes.c_int32, *[ctypes.c_void_p] * len(args))(ctypes.cast(f, ctypes.c_void_p).value)(*args)


@pytest.mark.parametrize("behind", [0, 1, 0x7F, 0xFF])
def test_the_first_structures_are_as_they_were(behind):
    L, c = kv.lib(), config_of(behind)
    out = (ctypes.c_size_t * (LAYOUT_WORDS + GUARD))(*([0xABCD] * (LAYOUT_WORDS + GUARD)))
    assert at(L.kvring_pages_get_layout, ctypes.addressof(c), ctypes.addressof(out)) == 0
    assert list(out[LAYOUT_WORDS:]) == [0xABCD] * GUARD
    lay = kv.kvring_pages_get_layout(kv.make_pages_config(32, 8, 128, 64, 1000, 16, 20, 512, layers=3))
    names = [f for f, _ in kv.KvringPagesLayout._fields_ if "block" not in f]
    assert list(out[:LAYOUT_WORDS]) == [getattr(lay, f) for f in names] and names[-1] == "total"
    # the config is taken by create as well, which then finds the buffer too small
    handle = ctypes.c_void_p()
    create = ctypes.CFUNCTYPE(ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                              ctypes.c_void_p)(ctypes.cast(L.kvring_pages_create, ctypes.c_void_p).value)
    assert create(ctypes.addressof(c), 0x1000, 1 << 10, None, ctypes.addressof(handle)) == 3


def test_options_are_taken_beside_the_config():
    L, c, word = kv.lib(), config_of(0xFF), ctypes.c_size_t
    out, k, v = (word * LAYOUT_WORDS)(), word(), word()
    call = lambda o: at(L.kvring_pages_get_layout_with, ctypes.addressof(c), o, ctypes.addressof(out), ctypes.addressof(k),  # noqa: E731
                        ctypes.addressof(v))
    assert call(None) == 0
    plain, n = list(out), 3 * 1000 * 8 * 4
    assert k.value == v.value
    o = kv.KvringPagesOptions(size=28)
    assert ctypes.sizeof(o) == 28 and call(ctypes.addressof(o)) == 0 and list(out) == plain
    o.scale_block = 16
    assert call(ctypes.addressof(o)) == 0
    up = (n + 255) // 256 * 256
    assert v.value - k.value == up and out[12] - plain[12] == 2 * up and list(out[:12]) == plain[:12]
    o.size = 24   # of another header
    assert call(ctypes.addressof(o)) == 1 and list(out) == [0] * LAYOUT_WORDS and (k.value, v.value) == (0, 0)
    o.size, handle = 28, ctypes.c_void_p()
    for opt, want in ((o, 3), (kv.KvringPagesOptions(size=28, scale_block=8), 1), (kv.KvringPagesOptions(scale_block=16), 1)):
        cfg = kv.make_pages_config(32, 8, 128, 64, 1000, 16, 20, 512, layers=3)
        assert L.kvring_pages_create_with(ctypes.byref(cfg), ctypes.byref(opt), 0x1000, 1 << 10, None, ctypes.byref(handle)) == want
