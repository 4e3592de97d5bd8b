"""Host-only checks of KvPages' binding: index tensors longer than the C calls'
32 bits count.  Nothing is allocated and nothing launched."""
import pytest
import torch

import ring_kv_cache_gb300 as kv


class Pages(kv.KvPages):
    """The binding alone; calls end in `counts`."""

    def __init__(self):
        self.device, self.counts = torch.device("meta"), []

    def _call(self, f, what, stream, *args):
        self.counts.append(args)
        raise kv.KvRingError(3, what)


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 1, 2 ** 33 + 7])
def test_requests_beyond_32_bits_do_not_wrap(n):
    kv.lib()
    p, x = Pages(), torch.empty(n, dtype=torch.int32, device="meta")
    with pytest.raises(kv.KvRingError):
        p.plan(x, 16)
    with pytest.raises(kv.KvRingError):
        p.plan(x, 16, rows=x)
    with pytest.raises(kv.KvRingError):
        p.release(x)
    most = 2 ** 31 - 1   # (more than any cache has requests, so the C calls refuse it)
    assert [a[2] for a in p.counts[:2]] == [most] * 2 and p.counts[2][1] == most
