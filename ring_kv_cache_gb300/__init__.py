"""Python binding of the kvring C ABI (``include/kvring.h``).

Argument marshalling only: every step of the cache's arithmetic runs in the
CUDA kernels of ``libkvring.so``.  PyTorch supplies device memory (one
``uint8`` buffer per ring, allocated once), streams and tensors.  There is
no CPU path: if the library is not built, or no sm_103a GPU is present,
calls raise.

The functions carry the C names (``kvring_create``, ``kvring_calibrate_scales``,
``kvring_write_frame``, ``kvring_delta_rotate``, ``kvring_attention``,
``kvring_export``); ``KvRing`` wraps them for one layer's cache.
"""
from __future__ import annotations

import ctypes
import os
import re
from collections import namedtuple

import torch

__all__ = [
    "KvRing", "KvRingError", "TO_OLDEST", "lib", "library_path", "header_functions",
    "kvring_required_bytes", "kvring_create", "kvring_destroy", "kvring_calibrate_scales",
    "kvring_write_frame", "kvring_delta_rotate", "kvring_attention", "kvring_attention_noalloc",
    "kvring_write_frames_many", "kvring_delta_rotate_many", "write_frames_many", "delta_rotate_many",
    "kvring_legacy_upkeep", "LegacyWindows", "kvring_project_write",
    "kvring_export",
    "kvring_status_string", "encode_e4m3", "STATE",
    "KvPages", "KvStep", "PAGES_STATE", "kvring_pages_get_layout", "kvring_pages_create", "kvring_pages_destroy",
]

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
HEADER = os.path.join(ROOT, "include", "kvring.h")

TO_OLDEST = -1
OUT_F32, OUT_BF16 = 0, 1
STATE = dict(head=0, n_valid=1, total_lo=2, total_hi=3, next_pos=4, calibrated=5, error=6,
             last_delta=7)
STATE_WORDS = 8
DEVERR_POSITION, DEVERR_TIMEOUT, DEVERR_DELTA = 1, 2, 4
PROJECT_WRITE, PROJECT_STORE_KV = 1, 2


class KvringConfig(ctypes.Structure):
    _fields_ = [
        ("num_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("capacity", ctypes.c_int32),
        ("max_tokens", ctypes.c_int32),
        ("max_position", ctypes.c_int32),
        ("max_kv_splits", ctypes.c_int32),
        ("attn_precision", ctypes.c_int32),
        ("pinned_prefix", ctypes.c_int32),
        ("rope_pairs_t", ctypes.c_int32),
        ("rope_pairs_y", ctypes.c_int32),
        ("rope_base", ctypes.c_double),
    ]


CACHE_E4M3, CACHE_BF16 = 0, 1
ROPE_ADJACENT, ROPE_HALVES = 0, 1
PAGES_STATE = dict(free=0, error=1, planned=2, requests=3, tokens=4, taken=5)
PAGES_STATE_WORDS = 8
PAGES_ERR_ROW, PAGES_ERR_TOKENS, PAGES_ERR_LENGTH, PAGES_ERR_PAGES = 1, 2, 4, 8
PAGES_ERR_COMMIT, PAGES_ERR_TABLE, PAGES_ERR_TIMEOUT = 16, 32, 64


class KvringPagesConfig(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in (
        "num_q_heads", "num_kv_heads", "head_dim", "num_layers", "page_size", "num_pages", "max_requests",
        "max_pages_per_request", "max_tokens", "cache_dtype", "rope_pairing", "reserved")] + [
        ("rope_base", ctypes.c_double)]


class KvringPagesLayout(ctypes.Structure):
    _fields_ = [(f, ctypes.c_size_t) for f in (
        "k_cache", "v_cache", "scales", "lengths", "tables", "free_pages", "state", "step_rows", "step_cu",
        "step_lengths", "positions", "slots", "total")]


class KvRingError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {kvring_status_string(status)} (status {status})")


_LIB = None


def library_path() -> str:
    return os.path.join(HERE, "libkvring.so")


def lib():
    """Load libkvring.so (built in-tree by ``ring_kv_cache_gb300.build``)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m ring_kv_cache_gb300.build`")
    L = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    cfgp = ctypes.POINTER(KvringConfig)
    sig = {
        "kvring_required_bytes": (sz, [cfgp]),
        "kvring_create": (i32, [cfgp, vp, sz, vp, ctypes.POINTER(vp)]),
        "kvring_destroy": (i32, [vp]),
        "kvring_calibrate_scales": (i32, [vp, vp, vp, vp, i32, vp]),
        "kvring_write_frame": (i32, [vp, vp, vp, vp, i32, vp]),
        "kvring_delta_rotate": (i32, [vp, i32, vp]),
        "kvring_write_frames_many": (i32, [vp, i32, vp, vp, vp, i32, vp]),
        "kvring_legacy_upkeep": (i32, [vp, vp, vp, vp, vp, vp, vp, i32, vp]),
        "kvring_delta_rotate_many": (i32, [vp, i32, i32, vp]),
        "kvring_attention": (i32, [vp, vp, vp, i32, vp, i32, vp]),
        "kvring_attention_noalloc": (i32, [vp, vp, vp, i32, vp, i32, vp]),
        "kvring_project_write": (i32, [vp, vp, vp, i32, vp, i32, vp, vp, i32, vp]),
        "kvring_export": (i32, [vp, vp, vp, vp, vp, vp, vp]),
        "kvring_pages_get_layout": (i32, [ctypes.POINTER(KvringPagesConfig), ctypes.POINTER(KvringPagesLayout)]),
        "kvring_pages_create": (i32, [ctypes.POINTER(KvringPagesConfig), vp, sz, vp, ctypes.POINTER(vp)]),
        "kvring_pages_destroy": (i32, [vp]),
        "kvring_pages_restore": (i32, [vp, vp, vp, vp, i32, vp]),
        "kvring_pages_set_scales": (i32, [vp, i32, vp, vp, vp]),
        "kvring_pages_plan": (i32, [vp, vp, vp, i32, i32, i32, vp]),
        "kvring_pages_commit": (i32, [vp, vp]),
        "kvring_pages_release": (i32, [vp, vp, i32, vp]),
        "kvring_pages_write": (i32, [vp, i32, vp, vp, vp, i64, i64, i64, vp, vp, ctypes.c_float, vp, i32, vp]),
        "kvring_pages_attention": (i32, [vp, i32, vp, i64, vp, i32, i32, i32, ctypes.c_float, vp]),
        "kvring_pages_debug_set_wait": (i32, [vp, i64, i32]),
        "kvring_debug_encode_e4m3": (i32, [vp, vp, i64, vp]),
        "kvring_debug_attention_levels": (i32, [vp, vp, vp]),
        "kvring_debug_set_attention_wait": (i32, [vp, i64, i32]),
        "kvring_debug_write_floor": (i32, [vp, i32, vp]),
        "kvring_debug_late_reads": (i64, []),
        "kvring_debug_attention_guess": (i32, [vp, i32]),
        "kvring_status_string": (ctypes.c_char_p, [i32]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _LIB = L
    return L


def header_functions() -> list[str]:
    """Names of the functions declared in include/kvring.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:[\w\s\*]+?)\b(kvring_\w+)\s*\(", text, re.M)))


def kvring_status_string(status: int) -> str:
    return lib().kvring_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != 0:
        raise KvRingError(status, what)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream_ptr(stream, device) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return s.cuda_stream


def _tokens(x: torch.Tensor, heads: int, dim: int, name: str, device=None) -> int:
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and x.device != device:
        raise ValueError(f"{name} is on {x.device}, the ring on {device}")
    if x.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16")
    if x.dim() != 3 or x.shape[1] != heads or x.shape[2] != dim:
        raise ValueError(f"{name} must have shape [n, {heads}, {dim}], got {tuple(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return x.shape[0]


def _positions(pos, n: int, name: str, three_d: bool = False, device=None):
    """Check a position tensor: int32 [n] (1-D RoPE) or [n, 3] = (t, y, x)."""
    if pos is None:
        if three_d:
            raise ValueError(f"{name}: 3-D RoPE needs explicit (t, y, x) positions")
        return None
    shape = (n, 3) if three_d else (n,)
    if not isinstance(pos, torch.Tensor) or not pos.is_cuda or pos.dtype != torch.int32 \
            or tuple(pos.shape) != shape or not pos.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA int32 tensor of shape {shape}")
    if device is not None and pos.device != device:
        raise ValueError(f"{name} is on {pos.device}, the ring on {device}")
    return pos


# ---------------------------------------------------------------------------
# C-named functions (marshalling only)
# ---------------------------------------------------------------------------
def make_config(heads, head_dim, capacity, max_tokens, max_position, rope_base=10000.0,
                max_kv_splits=16, attn_precision=0, pinned_prefix=0, rope3d=None) -> KvringConfig:
    pt, py = (0, 0) if rope3d is None else (int(rope3d[0]), int(rope3d[1]))
    return KvringConfig(int(heads), int(head_dim), int(capacity), int(max_tokens),
                        int(max_position), int(max_kv_splits), int(attn_precision),
                        int(pinned_prefix), pt, py, float(rope_base))


def kvring_required_bytes(cfg: KvringConfig) -> int:
    return int(lib().kvring_required_bytes(ctypes.byref(cfg)))


def kvring_create(cfg: KvringConfig, buf: torch.Tensor, stream=None) -> int:
    h = ctypes.c_void_p()
    _check(lib().kvring_create(ctypes.byref(cfg), buf.data_ptr(), buf.numel() * buf.element_size(),
                               _stream_ptr(stream, buf.device), ctypes.byref(h)), "kvring_create")
    return h.value


def kvring_destroy(handle: int) -> None:
    _check(lib().kvring_destroy(handle), "kvring_destroy")


def kvring_calibrate_scales(handle, k, v, pos, n, stream_ptr) -> None:
    _check(lib().kvring_calibrate_scales(handle, _ptr(k), _ptr(v), _ptr(pos), int(n), stream_ptr),
           "kvring_calibrate_scales")


def kvring_write_frame(handle, k, v, pos, n, stream_ptr) -> None:
    _check(lib().kvring_write_frame(handle, _ptr(k), _ptr(v), _ptr(pos), int(n), stream_ptr),
           "kvring_write_frame")


def kvring_delta_rotate(handle, delta, stream_ptr) -> None:
    _check(lib().kvring_delta_rotate(handle, int(delta), stream_ptr), "kvring_delta_rotate")


def _ptr_array(values):
    arr = (ctypes.c_void_p * len(values))()
    for i, x in enumerate(values):
        arr[i] = x
    return arr


def kvring_write_frames_many(handles, ks, vs, poss, n, stream_ptr) -> None:
    """Batched write: host arrays of ring handles and device pointers."""
    m = len(handles)
    pos_arr = None if poss is None else _ptr_array([_ptr(p) for p in poss])
    _check(lib().kvring_write_frames_many(_ptr_array(handles), m, _ptr_array([_ptr(k) for k in ks]),
                                          _ptr_array([_ptr(v) for v in vs]), pos_arr, int(n), stream_ptr),
           "kvring_write_frames_many")


def kvring_delta_rotate_many(handles, delta, stream_ptr) -> None:
    _check(lib().kvring_delta_rotate_many(_ptr_array(handles), len(handles), int(delta), stream_ptr),
           "kvring_delta_rotate_many")


def write_frames_many(rings, ks, vs, poss=None, stream=None) -> None:
    """kvring_write_frame on several rings of one shape in one launch."""
    if not rings or len(ks) != len(rings) or len(vs) != len(rings) or (poss is not None and len(poss) != len(rings)):
        raise ValueError("one k, v (and pos) per ring")
    r0 = rings[0]
    n = _tokens(ks[0], r0.H, r0.d, "k", r0.device)
    for i, r in enumerate(rings):
        if r.device != r0.device:
            raise ValueError("every ring must be on one device")
        if _tokens(ks[i], r.H, r.d, "k", r.device) != n or _tokens(vs[i], r.H, r.d, "v", r.device) != n:
            raise ValueError("every k and v must hold the same number of tokens")
        if poss is not None:
            _positions(poss[i], n, "pos", r.three_d, r.device)
        elif r.three_d:
            raise ValueError("3-D RoPE needs explicit (t, y, x) positions")
    with torch.cuda.device(r0.device):
        kvring_write_frames_many([r.handle for r in rings], ks, vs, poss, n, r0._s(stream))


def delta_rotate_many(rings, delta: int = TO_OLDEST, stream=None) -> None:
    """kvring_delta_rotate on several rings of one shape in one launch."""
    if not rings:
        raise ValueError("no rings")
    if any(r.device != rings[0].device for r in rings):
        raise ValueError("every ring must be on one device")
    with torch.cuda.device(rings[0].device):
        kvring_delta_rotate_many([r.handle for r in rings], delta, rings[0]._s(stream))


def kvring_legacy_upkeep(handle, wk_in, wv_in, wk_out, wv_out, k, v, n, stream_ptr) -> None:
    _check(lib().kvring_legacy_upkeep(handle, _ptr(wk_in), _ptr(wv_in), _ptr(wk_out), _ptr(wv_out), _ptr(k),
                                      _ptr(v), int(n), stream_ptr), "kvring_legacy_upkeep")


class LegacyWindows:
    """The two bf16 window buffer pairs the legacy upkeep alternates between."""

    def __init__(self, ring: "KvRing"):
        shape = (ring.C, ring.H, ring.d)
        self.ring = ring
        self.k = [torch.zeros(shape, dtype=torch.bfloat16, device=ring.device) for _ in range(2)]
        self.v = [torch.zeros(shape, dtype=torch.bfloat16, device=ring.device) for _ in range(2)]
        self.cur = 0

    def upkeep(self, k, v, stream=None) -> None:
        """One call of the original upkeep on `ring` with the frame (k, v)."""
        r = self.ring
        n = _tokens(k, r.H, r.d, "k", r.device)
        if _tokens(v, r.H, r.d, "v", r.device) != n:
            raise ValueError("k and v must hold the same number of tokens")
        a, b = self.cur, 1 - self.cur
        with torch.cuda.device(r.device):
            kvring_legacy_upkeep(r.handle, self.k[a], self.v[a], self.k[b], self.v[b], k, v, n, r._s(stream))
        self.cur = b

    def window(self):
        """The current (k, v) bf16 windows [capacity, H, d]."""
        return self.k[self.cur], self.v[self.cur]


def kvring_attention(handle, q, qpos, n_q, out, out_dtype, stream_ptr) -> None:
    _check(lib().kvring_attention(handle, _ptr(q), _ptr(qpos), int(n_q), _ptr(out), int(out_dtype),
                                  stream_ptr), "kvring_attention")


def kvring_attention_noalloc(handle, q, qpos, n_q, out, out_dtype, stream_ptr) -> None:
    _check(lib().kvring_attention_noalloc(handle, _ptr(q), _ptr(qpos), int(n_q), _ptr(out),
                                          int(out_dtype), stream_ptr), "kvring_attention_noalloc")


def kvring_project_write(handle, x, w, d_model, pos, n, q_out, kv_out, flags, stream_ptr) -> None:
    _check(lib().kvring_project_write(handle, _ptr(x), _ptr(w), int(d_model), _ptr(pos), int(n), _ptr(q_out),
                                      _ptr(kv_out), int(flags), stream_ptr), "kvring_project_write")


def kvring_export(handle, k_out, v_out, scales, slot_pos, state, stream_ptr) -> None:
    _check(lib().kvring_export(handle, _ptr(k_out), _ptr(v_out), _ptr(scales), _ptr(slot_pos),
                               _ptr(state), stream_ptr), "kvring_export")


def late_reads() -> int:
    """How many write and attention calls so far read their frame or queries
    after waiting for the preceding kernel, because the library's previous
    kernel on their stream writes a buffer overlapping them."""
    return int(lib().kvring_debug_late_reads())


def encode_e4m3(x: torch.Tensor, stream=None) -> torch.Tensor:
    """E4M3 codes of a CUDA float32 tensor, with the kernels' conversion (test support)."""
    if not x.is_cuda or x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA float32 tensor")
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check(lib().kvring_debug_encode_e4m3(x.data_ptr(), out.data_ptr(), x.numel(),
                                          _stream_ptr(stream, x.device)), "kvring_debug_encode_e4m3")
    return out


# ---------------------------------------------------------------------------
class KvRing:
    """One layer's rolling FP8 attention cache on one CUDA device (the
    current one unless ``device`` names another).  Every call runs with that
    device current and takes tensors on it.  The ring's buffer is freed with
    the object: keep it alive until the work enqueued on it has completed."""

    def __init__(self, heads: int, head_dim: int, capacity: int, max_tokens: int,
                 max_position: int, rope_base: float = 10000.0, max_kv_splits: int = 16,
                 attn_precision: int = 0, device=None, stream=None, pinned_prefix: int = 0,
                 rope3d=None):
        if not torch.cuda.is_available():
            raise RuntimeError("KvRing needs a CUDA device")
        d = torch.device(device) if device is not None else torch.device("cuda")
        if d.type != "cuda":
            raise ValueError("KvRing needs a CUDA device")
        self.device = d if d.index is not None else torch.device("cuda", torch.cuda.current_device())
        self.H, self.d, self.C = int(heads), int(head_dim), int(capacity)
        self.max_tokens = int(max_tokens)
        self.P = int(pinned_prefix)
        self.three_d = rope3d is not None
        self.cfg = make_config(heads, head_dim, capacity, max_tokens, max_position, rope_base,
                               max_kv_splits, attn_precision, pinned_prefix, rope3d)
        n = kvring_required_bytes(self.cfg)
        if n == 0:
            raise ValueError("invalid kvring config")
        self.nbytes = n
        with torch.cuda.device(self.device):
            self.buf = torch.empty(n, dtype=torch.uint8, device=self.device)
            self.handle = kvring_create(self.cfg, self.buf, stream)

    def _s(self, stream) -> int:
        return _stream_ptr(stream, self.device)

    def calibrate(self, k, v, pos=None, stream=None) -> None:
        n = _tokens(k, self.H, self.d, "k", self.device)
        if _tokens(v, self.H, self.d, "v", self.device) != n:
            raise ValueError("k and v must hold the same number of tokens")
        pos = _positions(pos, n, "pos", self.three_d, self.device)
        with torch.cuda.device(self.device):
            kvring_calibrate_scales(self.handle, k, v, pos, n, self._s(stream))

    def write(self, k, v, pos=None, stream=None) -> None:
        n = _tokens(k, self.H, self.d, "k", self.device)
        if _tokens(v, self.H, self.d, "v", self.device) != n:
            raise ValueError("k and v must hold the same number of tokens")
        pos = _positions(pos, n, "pos", self.three_d, self.device)
        with torch.cuda.device(self.device):
            kvring_write_frame(self.handle, k, v, pos, n, self._s(stream))

    def delta_rotate(self, delta: int = TO_OLDEST, stream=None) -> None:
        with torch.cuda.device(self.device):
            kvring_delta_rotate(self.handle, delta, self._s(stream))

    def attention(self, q, qpos=None, out=None, out_dtype=torch.float32, stream=None) -> torch.Tensor:
        n = _tokens(q, self.H, self.d, "q", self.device)
        if out is None:
            out = torch.empty((n, self.H, self.d), dtype=out_dtype, device=self.device)
        if out.dtype not in (torch.float32, torch.bfloat16) or tuple(out.shape) != (n, self.H, self.d) \
                or not out.is_contiguous() or not out.is_cuda or out.device != self.device:
            raise ValueError("out must be a contiguous float32/bfloat16 tensor [n_q, H, d] on the ring's device")
        qpos = _positions(qpos, n, "qpos", self.three_d, self.device)
        with torch.cuda.device(self.device):
            kvring_attention(self.handle, q, qpos, n, out,
                             OUT_BF16 if out.dtype == torch.bfloat16 else OUT_F32, self._s(stream))
        return out

    def project_write(self, x, w, pos=None, write=True, store_kv=False, q_out=None, kv_out=None,
                      stream=None):
        """QKV projection of one frame with the cache write fused in
        (kvring_project_write): x bf16 [n, d_model], w bf16 [3 H d, d_model]
        (a linear layer's weight); returns (q_out bf16 [n, H, d], kv_out bf16
        [2, n, H, d] or None).  With ``write`` the keys and values enter the
        ring as kvring_write_frame would write them; ``store_kv`` also returns
        them (e.g. to calibrate a session from its first frame)."""
        for t, name in ((x, "x"), (w, "w")):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 2 \
                    or not t.is_contiguous() or t.device != self.device:
                raise ValueError(f"{name} must be a contiguous 2-D bfloat16 tensor on {self.device}")
        n, dm = x.shape
        if dm < 64 or dm % 64:
            raise ValueError("d_model must be a positive multiple of 64")
        if tuple(w.shape) != (3 * self.H * self.d, dm):
            raise ValueError(f"w must have shape [{3 * self.H * self.d}, {dm}], got {tuple(w.shape)}")
        if pos is not None or (write and self.three_d):
            pos = _positions(pos, n, "pos", self.three_d, self.device)
        if q_out is None:
            q_out = torch.empty((n, self.H, self.d), dtype=torch.bfloat16, device=self.device)
        _tokens(q_out, self.H, self.d, "q_out", self.device)
        if store_kv:
            if kv_out is None:
                kv_out = torch.empty((2, n, self.H, self.d), dtype=torch.bfloat16, device=self.device)
            if kv_out.dtype != torch.bfloat16 or tuple(kv_out.shape) != (2, n, self.H, self.d) \
                    or not kv_out.is_contiguous() or kv_out.device != self.device:
                raise ValueError("kv_out must be a contiguous bfloat16 tensor [2, n, H, d] on the ring's device")
        flags = (PROJECT_WRITE if write else 0) | (PROJECT_STORE_KV if store_kv else 0)
        with torch.cuda.device(self.device):
            kvring_project_write(self.handle, x, w, dm, pos, n, q_out, kv_out if store_kv else None, flags,
                                 self._s(stream))
        return q_out, (kv_out if store_kv else None)

    def export(self, stream=None) -> dict:
        """Device copies of the cache, scales, positions and state (stream-ordered)."""
        dev = self.device
        k = torch.empty((self.H, self.C, self.d), dtype=torch.uint8, device=dev)
        v = torch.empty_like(k)
        scales = torch.empty(4 * self.H, dtype=torch.float32, device=dev)
        slot_pos = torch.empty(self.C, dtype=torch.int32, device=dev)
        state = torch.empty(STATE_WORDS, dtype=torch.int32, device=dev)
        with torch.cuda.device(dev):
            kvring_export(self.handle, k, v, scales, slot_pos, state, self._s(stream))
        return dict(k=k, v=v, scales=scales, slot_pos=slot_pos, state=state)

    def levels(self, stream=None) -> torch.Tensor:
        qt = (self.max_tokens + 127) // 128
        out = torch.empty((qt, self.H), dtype=torch.int32, device=self.device)
        with torch.cuda.device(self.device):
            _check(lib().kvring_debug_attention_levels(self.handle, out.data_ptr(), self._s(stream)),
                   "kvring_debug_attention_levels")
        return out

    def write_floor(self, n: int, stream=None) -> None:
        """Measurement support: the write's fixed cost for n tokens, no data
        (see the C header); the ring is left unchanged."""
        with torch.cuda.device(self.device):
            _check(lib().kvring_debug_write_floor(self.handle, int(n), self._s(stream)),
                   "kvring_debug_write_floor")

    def set_attention_guess(self, wrong: bool = False) -> None:
        """Test support: make the attention's early guess of the default
        query positions wrong on purpose (kvring_debug_attention_guess)."""
        _check(lib().kvring_debug_attention_guess(self.handle, int(bool(wrong))), "kvring_debug_attention_guess")

    def set_attention_wait(self, limit_ns: int = 1_000_000_000, stall: bool = False) -> None:
        """Test support: the attention kernel's wait limit, and a stall that
        makes its first wait give up on purpose (see the C header)."""
        _check(lib().kvring_debug_set_attention_wait(self.handle, int(limit_ns), int(bool(stall))),
               "kvring_debug_set_attention_wait")

    def close(self) -> None:
        if getattr(self, "handle", None):
            kvring_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# The paged cache
# ---------------------------------------------------------------------------
def _i32(x) -> int:
    """An int argument, kept in range where ctypes would wrap it."""
    x = int(x)
    return x if -(1 << 31) <= x < 1 << 31 else (-1 if x < 0 else (1 << 31) - 1)


def make_pages_config(q_heads, kv_heads, head_dim, page_size, num_pages, max_requests, max_pages_per_request,
                      max_tokens, layers=1, cache_dtype=CACHE_E4M3, rope_pairing=ROPE_ADJACENT,
                      rope_base=10000.0) -> KvringPagesConfig:
    return KvringPagesConfig(*map(_i32, (q_heads, kv_heads, head_dim, layers, page_size, num_pages, max_requests,
                                         max_pages_per_request, max_tokens, cache_dtype, rope_pairing, 0)),
                             float(rope_base))


def _empty_on(stream, shape, dtype, device) -> torch.Tensor:
    """A new tensor that ``stream`` (None: the current one) may write: memory
    of that stream's own, which no work on another may still be using, and
    which goes back to it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def kvring_pages_get_layout(cfg: KvringPagesConfig) -> KvringPagesLayout:
    lay = KvringPagesLayout()
    _check(lib().kvring_pages_get_layout(ctypes.byref(cfg), ctypes.byref(lay)), "kvring_pages_get_layout")
    return lay


def kvring_pages_create(cfg: KvringPagesConfig, buf: torch.Tensor, stream=None) -> int:
    h = ctypes.c_void_p()
    _check(lib().kvring_pages_create(ctypes.byref(cfg), buf.data_ptr(), buf.numel() * buf.element_size(),
                                     _stream_ptr(stream, buf.device), ctypes.byref(h)), "kvring_pages_create")
    return h.value


def kvring_pages_destroy(handle: int) -> None:
    _check(lib().kvring_pages_destroy(handle), "kvring_pages_destroy")


# What a plan made, as views of the cache's own buffer (valid until the next
# plan): cu [requests + 1], lengths [requests] with the new tokens, positions
# and slots [num_tokens] (slot -1: padding).
KvStep = namedtuple("KvStep", "cu lengths positions slots")


class KvPages:
    """A paged cache of every layer of a model for many requests, on one CUDA
    device (the current one unless ``device`` names another).

    A step: ``plan`` the new tokens of its requests, then for every layer
    ``write`` and ``attention``, then ``commit``; ``release`` ends requests.
    All of it runs on the device and can be captured in a CUDA graph.  Calls
    on one object must be ordered (one stream, or events); graphs that use
    one share its plan and workspace.  Every call runs with the object's
    device current and takes tensors on it.  A tensor that a call with
    ``stream`` makes belongs to that stream.  The object's buffer is freed with
    it: keep it alive until the work enqueued on it has completed.
    """

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, page_size: int, num_pages: int, max_requests: int,
                 max_request_tokens: int, max_tokens: int, layers: int = 1, cache_dtype=torch.float8_e4m3fn,
                 rope_pairing: str = "adjacent", rope_base: float = 10000.0, device=None, stream=None):
        if not torch.cuda.is_available():
            raise RuntimeError("KvPages needs a CUDA device")
        d = torch.device(device) if device is not None else torch.device("cuda")
        if d.type != "cuda":
            raise ValueError("KvPages needs a CUDA device")
        if cache_dtype not in (torch.float8_e4m3fn, torch.bfloat16):
            raise ValueError("cache_dtype must be float8_e4m3fn or bfloat16")
        if rope_pairing not in ("adjacent", "halves"):
            raise ValueError("rope_pairing must be 'adjacent' or 'halves'")
        self.device = d if d.index is not None else torch.device("cuda", torch.cuda.current_device())
        self.Hq, self.Hkv, self.d, self.P = int(q_heads), int(kv_heads), int(head_dim), int(page_size)
        self.L, self.num_pages, self.R = int(layers), int(num_pages), int(max_requests)
        self.W = -(-int(max_request_tokens) // max(1, self.P))
        self.max_tokens, self.cache_dtype = int(max_tokens), cache_dtype
        self.cfg = make_pages_config(q_heads, kv_heads, head_dim, page_size, num_pages, max_requests, self.W,
                                     max_tokens, layers, CACHE_E4M3 if cache_dtype == torch.float8_e4m3fn
                                     else CACHE_BF16, ROPE_HALVES if rope_pairing == "halves" else ROPE_ADJACENT,
                                     rope_base)
        try:
            self.layout = kvring_pages_get_layout(self.cfg)
        except KvRingError:
            raise ValueError("invalid paged-cache config") from None
        self.nbytes = int(self.layout.total)
        with torch.cuda.device(self.device):
            self.buf = _empty_on(stream, (self.nbytes,), torch.uint8, self.device)
            self.handle = kvring_pages_create(self.cfg, self.buf, stream)
        lay = self.layout
        self.lengths = self._ints(lay.lengths, self.R)
        self.tables = self._ints(lay.tables, self.R * self.W).view(self.R, self.W)
        self.free_pages = self._ints(lay.free_pages, self.num_pages)
        self.state = self._ints(lay.state, PAGES_STATE_WORDS)
        self._cu, self._klen = self._ints(lay.step_cu, self.R + 1), self._ints(lay.step_lengths, self.R)
        self._pos, self._slots = self._ints(lay.positions, self.max_tokens), self._ints(lay.slots, self.max_tokens)
        self._steps, self._caches, self._index = {}, {}, self.device.index

    def _ints(self, off: int, n: int) -> torch.Tensor:
        return self.buf[off:off + 4 * n].view(torch.int32)

    def _call(self, f, what: str, stream, *args) -> None:
        """A library call on the object's device and the given (or its current) stream."""
        s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(self._index)
        if torch.cuda.current_device() == self._index:
            _check(f(self.handle, *args, s), what)
        else:
            with torch.cuda.device(self.device):
                _check(f(self.handle, *args, s), what)

    def _cache(self, off: int, layer: int) -> torch.Tensor:
        if (off, layer) not in self._caches:
            self._caches[off, layer] = self._cache_view(off, layer)
        return self._caches[off, layer]

    def _cache_view(self, off: int, layer: int) -> torch.Tensor:
        if not 0 <= layer < self.L:
            raise ValueError(f"layer must be in [0, {self.L})")
        shape = (self.num_pages, self.Hkv, self.P, self.d)
        n = self.num_pages * self.Hkv * self.P * self.d * self.cache_dtype.itemsize
        return self.buf[off + layer * n:off + (layer + 1) * n].view(self.cache_dtype).view(shape)

    def k_cache(self, layer: int = 0) -> torch.Tensor:
        """The layer's keys [num_pages, Hkv, page_size, d], a view of the buffer."""
        return self._cache(self.layout.k_cache, layer)

    def v_cache(self, layer: int = 0) -> torch.Tensor:
        """The layer's values [num_pages, Hkv, page_size, d], a view of the buffer."""
        return self._cache(self.layout.v_cache, layer)

    def _int_arg(self, x, name: str, shape=None):
        if not isinstance(x, torch.Tensor) or x.device != self.device or x.dtype != torch.int32 \
                or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor on {self.device}")
        if (shape is None and x.dim() != 1) or (shape is not None and tuple(x.shape) != shape):
            raise ValueError(f"{name} must have shape {shape or '[n]'}, got {tuple(x.shape)}")
        return x

    def restore(self, lengths, tables, free_pages, stream=None) -> None:
        """Take over a state: int32 lengths [max_requests], block tables
        [max_requests, pages per request] and the stack of free pages [n]."""
        self._int_arg(lengths, "lengths", (self.R,))
        self._int_arg(tables, "tables", (self.R, self.W))
        n = self._int_arg(free_pages, "free_pages").numel()
        if n > self.num_pages:
            raise ValueError(f"free_pages holds {n} pages, the cache {self.num_pages}")
        self._call(_LIB.kvring_pages_restore, "kvring_pages_restore", stream, lengths.data_ptr(), tables.data_ptr(),
                   free_pages.data_ptr() if n else None, n)

    def set_scales(self, layer: int, scale_k, scale_v, stream=None) -> None:
        """Per-head scales (float32 [Hkv]) of one layer of an E4M3 cache."""
        for t, name in ((scale_k, "scale_k"), (scale_v, "scale_v")):
            if not isinstance(t, torch.Tensor) or t.device != self.device or t.dtype != torch.float32 \
                    or tuple(t.shape) != (self.Hkv,) or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 tensor [{self.Hkv}] on {self.device}")
        self._call(_LIB.kvring_pages_set_scales, "kvring_pages_set_scales", stream, _i32(layer), scale_k.data_ptr(),
                   scale_v.data_ptr())

    def plan(self, new_tokens, num_tokens: int, rows=None, max_new: int | None = None, stream=None) -> KvStep:
        """Plan a step: request i (row ``rows[i]``, or row i) gets
        ``new_tokens[i]`` tokens; ``num_tokens`` is the token count of the
        step's tensors (at least the sum), ``max_new`` a bound on every
        ``new_tokens[i]``.  Both index tensors are int32 on the device."""
        n = self._int_arg(new_tokens, "new_tokens").numel()
        if rows is not None:
            self._int_arg(rows, "rows", (n,))
        num_tokens = _i32(num_tokens)
        self._call(_LIB.kvring_pages_plan, "kvring_pages_plan", stream, _ptr(rows), new_tokens.data_ptr(), n, num_tokens,
                   num_tokens if max_new is None else _i32(max_new))
        step = self._steps.get((n, num_tokens))
        if step is None:
            if len(self._steps) >= 256:
                self._steps.clear()
            step = self._steps[(n, num_tokens)] = KvStep(self._cu[:n + 1], self._klen[:n], self._pos[:num_tokens],
                                                         self._slots[:num_tokens])
        return step

    def commit(self, stream=None) -> None:
        """Make the last plan final: the lengths and the free list."""
        self._call(_LIB.kvring_pages_commit, "kvring_pages_commit", stream)

    def release(self, rows, stream=None) -> None:
        """End the requests in ``rows`` (int32): their pages become free."""
        n = self._int_arg(rows, "rows").numel()
        self._call(_LIB.kvring_pages_release, "kvring_pages_release", stream, rows.data_ptr(), n)

    def _heads(self, x, heads: int, name: str):
        """Check bf16 [n, heads, d] with whole rows of heads (a slice of a
        packed projection output is one); returns n and the token stride."""
        if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or x.device != self.device:
            raise ValueError(f"{name} must be a bfloat16 tensor on {self.device}")
        shape, row = x.shape, heads * self.d
        if len(shape) != 3 or shape[1] != heads or shape[2] != self.d:
            raise ValueError(f"{name} must have shape [n, {heads}, {self.d}], got {tuple(shape)}")
        n = shape[0]
        st, sh, s1 = x.stride()
        if s1 != 1 or (heads > 1 and sh != self.d) or (n > 1 and st < row):
            raise ValueError(f"{name}: the heads of a token must be contiguous, and tokens must not overlap")
        return n, st if n > 1 else row

    def _result(self, x, n: int, name: str, stream):
        if x is None:
            return _empty_on(stream, (n, self.Hq, self.d), torch.bfloat16, self.device)
        if self._heads(x, self.Hq, name) != (n, self.Hq * self.d):
            raise ValueError(f"{name} must be contiguous, [{n}, {self.Hq}, {self.d}]")
        return x

    def write(self, layer: int, q, k, v, q_norm=None, k_norm=None, eps: float = 1e-6, q_out=None,
              stream=None) -> torch.Tensor:
        """Head norms (where weights bf16 [d] are given), RoPE and the write of
        the planned tokens' keys and values; returns the rotated queries
        (bf16 [n, Hq, d]).  Rows of ``q_out`` past the plan's tokens are left
        as they were (undefined in a new tensor)."""
        n, qs = self._heads(q, self.Hq, "q")
        nk, ks = self._heads(k, self.Hkv, "k")
        nv, vs = self._heads(v, self.Hkv, "v")
        if nk != n or nv != n:
            raise ValueError("q, k and v must hold the same number of tokens")
        for t, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
            if t is not None and (not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16
                                  or t.device != self.device or t.shape != (self.d,) or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous bfloat16 tensor [{self.d}] on {self.device}")
        q_out = self._result(q_out, n, "q_out", stream)
        self._call(_LIB.kvring_pages_write, "kvring_pages_write", stream, _i32(layer), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                   qs, ks, vs, _ptr(q_norm), _ptr(k_norm), float(eps), q_out.data_ptr(), n)
        return q_out

    def attention(self, layer: int, q, out=None, causal: bool = True, window: int = 0, scale: float = 0.0,
                  stream=None) -> torch.Tensor:
        """Attention of the planned tokens' queries (rotated, bf16 [n, Hq, d])
        over their requests' cached tokens, the new ones included.  ``window``
        limits a causal query to its last ``window`` tokens; ``scale`` 0 means
        1/sqrt(d).  Rows of ``out`` past the plan's tokens are left as they
        were (undefined in a new tensor)."""
        n, qs = self._heads(q, self.Hq, "q")
        out = self._result(out, n, "out", stream)
        self._call(_LIB.kvring_pages_attention, "kvring_pages_attention", stream, _i32(layer), q.data_ptr(), qs, out.data_ptr(),
                   n, 1 if causal else 0, _i32(window), float(scale))
        return out

    def set_wait(self, limit_ns: int = 1_000_000_000, stall: bool = False) -> None:
        """Test support: the attention kernels' wait limit, and a stall that
        makes their first wait give up on purpose (see the C header)."""
        _check(lib().kvring_pages_debug_set_wait(self.handle, int(limit_ns), int(bool(stall))),
               "kvring_pages_debug_set_wait")

    def close(self) -> None:
        if getattr(self, "handle", None):
            kvring_pages_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
