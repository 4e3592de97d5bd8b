"""Host-only checks of residual_norm's binding: row counts that the C config's
32 bits do not hold.  Nothing is allocated and nothing launched."""
import pytest
import torch

import ring_kv_cache_gb300 as kv

BF = torch.bfloat16


class OnGpu(torch.Tensor):
    """A tensor without memory that says it is on cuda:0."""
    is_cuda = True

    def get_device(self):
        return 0


def tensor(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta").as_subclass(OnGpu)


@pytest.fixture(autouse=True)
def no_call(monkeypatch):
    def launched(*_):
        raise AssertionError("the call went through")

    monkeypatch.setattr(kv, "lib", launched)
    monkeypatch.setattr(kv, "_empty_on", lambda s, shape, dtype, device: tensor(*shape, dtype=dtype))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 33 + 1])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_more_rows_than_32_bits_are_refused(n, dtype):
    h = tensor(n, 8, dtype=dtype)
    for args in ((h,), (h, tensor(n, 8))):
        with pytest.raises(ValueError, match="rows"):
            kv.residual_norm(*args)


@pytest.mark.parametrize("m", [2 ** 31, 2 ** 32 + 1, 2 ** 32 + 5])
@pytest.mark.parametrize("which", ["gate", "scale", "shift"])
def test_more_table_rows_than_32_bits_are_refused(m, which):
    for rows in (None, tensor(5, dtype=torch.int32)):
        with pytest.raises(ValueError, match="rows"):
            kv.residual_norm(tensor(5, 8), tensor(5, 8), mod_rows=rows, **{which: tensor(m, 8)})


def test_what_32_bits_hold_goes_through():
    n = 2 ** 31 - 1
    for args, kw in (((tensor(n, 8), tensor(n, 8)), {}),
                     ((tensor(5, 8), tensor(5, 8)), dict(gate=tensor(n, 8), mod_rows=tensor(5, dtype=torch.int32)))):
        with pytest.raises(AssertionError, match="went through"):
            kv.residual_norm(*args, **kw)
