"""Host-only checks of kvring_residual_norm: what the C entry refuses before it
launches anything.  The pointers are never followed."""
import ctypes

import pytest

import ring_kv_cache_gb300 as kv

H, Y, GATE, SCALE, SHIFT, INDEX, POST, W, HO, XO = [(i + 1) << 28 for i in range(10)]   # far apart, 16-byte aligned


def config(**kw):
    base = dict(num_tokens=9, width=64, stream_dtype=kv.OUT_F32, mod_dtype=kv.OUT_BF16, mod_rows=3, post_norm=1, norm=2,
                reserved=0, h_stride=64, y_stride=64, mod_stride=192, h_out_stride=64, x_out_stride=64, eps=1e-6,
                residual_scale=1.0)
    return kv.KvringNormConfig(*{**base, **kw}.values())


def call(cfg=None, h=H, y=Y, gate=GATE, scale=SCALE, shift=SHIFT, index=INDEX, post=POST, w=W, ho=HO, xo=XO, **kw):
    cfg = config(**kw) if cfg is None else cfg
    return kv.lib().kvring_residual_norm(ctypes.byref(cfg), h, y, gate, scale, shift, index, post, w, ho, xo, None)


@pytest.mark.parametrize("field,value", [
    ("num_tokens", 0), ("num_tokens", -1), ("width", 0), ("width", 12), ("width", 16392), ("stream_dtype", 2),
    ("mod_dtype", -1), ("mod_rows", 0), ("post_norm", 3), ("norm", -1), ("reserved", 1), ("h_stride", 56),
    ("h_stride", 68), ("y_stride", 0), ("mod_stride", 100), ("h_out_stride", -64), ("x_out_stride", 1 << 29),
    ("eps", -1.0), ("eps", float("nan")), ("eps", float("inf")), ("residual_scale", float("nan"))])
def test_bad_configs_are_refused(field, value):
    assert call(**{field: value}) == 1


@pytest.mark.parametrize("what", [
    dict(h=None), dict(h=H + 8), dict(y=Y + 2), dict(gate=GATE + 4), dict(index=INDEX + 2), dict(ho=HO + 8), dict(xo=XO + 8),
    dict(y=None), dict(y=None, gate=None), dict(y=None, gate=None, post=None), dict(y=None, gate=None, post=None, post_norm=0),
    dict(post_norm=0), dict(norm=0), dict(xo=None), dict(norm=0, xo=None), dict(norm=0, xo=None, w=None),
    dict(gate=None, scale=None, shift=None), dict(index=None), dict(index=None, mod_rows=8),
    dict(ho=None, xo=None, norm=0, w=None, scale=None, shift=None)])
def test_arguments_that_say_two_things_are_refused(what):
    assert call(**what) == 1


@pytest.mark.parametrize("what", [
    dict(ho=H + 256), dict(ho=H, h_out_stride=128), dict(xo=H), dict(xo=HO), dict(xo=HO + 64 * 9 * 4 - 16), dict(xo=Y),
    dict(ho=Y), dict(ho=GATE), dict(xo=SCALE + 128), dict(xo=SHIFT + 2 * 192 * 2), dict(xo=INDEX), dict(xo=W), dict(ho=POST)])
def test_results_over_arguments_are_refused(what):
    assert call(**what) == 1


def test_a_null_config_is_refused():
    assert kv.lib().kvring_residual_norm(None, H, Y, GATE, SCALE, SHIFT, INDEX, POST, W, HO, XO, None) == 1
