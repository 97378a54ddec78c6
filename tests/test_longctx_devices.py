"""Workspaces that the long-context calls make for themselves are sized on the
tensors' device, not on the current one, which may have other SMs (CPU only,
with a fake of the device calls)."""
import contextlib

import pytest
import torch


@pytest.mark.parametrize("current", [0, 1])
def test_scratch_is_sized_on_the_tensors_device(monkeypatch, current):
    from paged_kv_decode_04_gb300 import build
    build.build()
    from paged_kv_decode_04_gb300 import binding as B
    now = [current]

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], index
        yield
        now[0] = before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(B, "_new", lambda n, dtype, index, stream: torch.empty(n, dtype=dtype))
    _, _, size = B._scratch(None, lambda: {0: 100, 1: 300}[now[0]], 1, None)
    assert size == 300 and now[0] == current


def test_scratch_of_nothing_and_of_the_callers(monkeypatch):
    from paged_kv_decode_04_gb300 import binding as B
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    assert B._scratch(None, lambda: 0, 0, None) == (None, None, 0)
    with pytest.raises(ValueError, match="workspace"):
        B._scratch(torch.empty(16, dtype=torch.uint8), lambda: 0, 0, None)
