"""Which device the decode operators' calls go to (no GPU: a torch and a library
that only note what they are asked for).  The handle of a default stream is 0 on
every device, and a launch on it goes to the current one."""
import contextlib

import pytest

from weight_only_block_amd import qgemv as Q

torch = pytest.importorskip("torch")


class Tensor:
    """A contiguous GPU tensor's outside."""
    device = type("device", (), {"type": "cuda"})()

    def __init__(self, dtype, shape, where):
        self.dtype, self.shape, self.where = dtype, torch.Size(shape), where

    def stride(self, dim=None):
        steps = [1]
        for n in self.shape[:0:-1]:
            steps.insert(0, steps[0] * n)
        return tuple(steps) if dim is None else steps[dim]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def get_device(self):
        return self.where

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def calls(monkeypatch):
    """(entry, device current at the call) of every call; device 0 is current."""
    log, current = [], [0]
    kinds = Q._dtypes()
    monkeypatch.setattr(Q, "_DT", kinds)

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        try:
            yield
        finally:
            current[0] = before

    monkeypatch.setattr(kinds, "current_device", staticmethod(lambda: current[0]), raising=False)
    monkeypatch.setattr(kinds, "current_stream", staticmethod(lambda index: 0))
    monkeypatch.setattr(kinds, "device", staticmethod(device), raising=False)

    class Library:
        def __getattr__(self, name):
            return lambda *args: log.append((name, current[0])) or 0

    monkeypatch.setattr(Q, "lib", Library)
    return log, current


@pytest.mark.parametrize("where", [0, 1])
@pytest.mark.parametrize("stream", [None, 0])
def test_calls_go_to_the_tensors_device(calls, where, stream):
    log, current = calls
    t = lambda dtype, *shape: Tensor(dtype, shape, where)
    bf16, f32, i32, i64, u8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
    cache = Q.KVCache.__new__(Q.KVCache)
    cache.kv_heads, cache.page_size, cache.head_dim, cache.device, cache._ref = 2, 16, 64, where, 0
    rope = Q.Rope.__new__(Q.Rope)
    rope._ref = 0
    assert Q.rope_append(cache, rope, t(f32, 3, 4, 64), t(f32, 3, 2, 64), t(f32, 3, 2, 64), t(i32, 3), t(i64, 3),
                         t(bf16, 3, 4, 64), stream=stream) == 0
    assert Q.kv_read(cache, t(i64, 3), t(f32, 3, 2, 64), t(f32, 3, 2, 64), stream=stream) == 0
    assert Q.paged_attention(cache, t(bf16, 3, 4, 64), t(bf16, 3, 4, 64), t(i32, 4), t(i32, 3), t(i32, 3, 5), t(u8, 4096), 1, 80,
                             stream=stream) == 0
    assert Q.sample_f32(t(f32, 3, 100), t(f32, 3), t(i32, 3), t(u8, 4096), stream=stream) == 0
    assert log == [(name, where) for name in ("qg_rope_append", "qg_kv_read", "qg_paged_attention", "qg_sample_f32")]
    assert current == [0]
