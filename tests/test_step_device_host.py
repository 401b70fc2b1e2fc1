"""The workspace query of cross attention asks the cache's device (no GPU: the
device switch is watched from a stand-in)."""

import ctypes

import torch

import paged_kv_cache_145_gb300 as pkv
from tests.test_abi import fake_cache


class Cache:
    """What the query needs of a PagedKVCache on the second of two devices."""
    device = torch.device("cuda", 1)

    def __init__(self):
        self._c = fake_cache()
        self.ref = ctypes.byref(self._c)


def watch(monkeypatch, current):
    entered, now = [], [current]

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)
            now.append(self.device.index)

        def __exit__(self, *args):
            entered.append(None)
            now.pop()

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "device", Device)
    return entered


def test_the_plan_is_made_on_the_caches_device(monkeypatch):
    entered = watch(monkeypatch, 0)
    assert pkv.paged_attention_cross_workspace_bytes(Cache(), 4, 2, 4, 3, 100) >= 0
    assert entered == [Cache.device, None]


def test_the_current_device_is_not_entered_again(monkeypatch):
    entered = watch(monkeypatch, 1)
    assert pkv.paged_attention_cross_workspace_bytes(Cache(), 4, 2, 4, 3, 100) >= 0
    assert entered == []
