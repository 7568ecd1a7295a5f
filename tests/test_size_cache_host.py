"""Sizes that the library gives by the device's number of SMs are kept by device. CPU only."""
import pytest

from route_permute_grouped_gb300 import ops


class _Lib:
    """The library as it answers on devices of 100 SMs and of 200."""

    def __init__(self):
        self.device, self.asked = 0, 0

    def _sized(self, *_):
        self.asked += 1
        return 256 + 1000 * (1 + self.device)

    moe_norm_workspace_bytes = moe_few_workspace_bytes = _sized


@pytest.fixture
def lib(monkeypatch):
    fake = _Lib()
    monkeypatch.setattr(ops, "lib", lambda: fake)
    monkeypatch.setattr(ops, "_current_device", lambda: fake.device)
    monkeypatch.setattr(ops, "_size_cache", {})
    monkeypatch.setattr(ops, "_norm_plans", {})
    return fake


def test_a_size_is_asked_once_a_device(lib):
    cfg = ops.make_config(4, 128, 8, 2, 128)
    for _ in range(2):
        for lib.device in (0, 1):
            assert ops.few_workspace(cfg, device="cpu").numel() == 1256 + 1000 * lib.device
    assert lib.asked == 2


def test_a_norm_plan_is_made_once_a_device(lib):
    cfg = ops.make_norm_config(4, 128)
    for _ in range(2):
        for lib.device in (0, 1):
            assert ops._norm_plan(cfg).nbytes == ops.norm_workspace(cfg, device="cpu").numel() == 1256 + 1000 * lib.device
    assert lib.asked == 2


@pytest.mark.parametrize("error", [RuntimeError, AssertionError])
def test_without_a_device_sizes_are_still_given(lib, monkeypatch, error):
    def none():
        raise error("no device")
    monkeypatch.setattr(ops, "_current_device", none)
    assert ops.norm_workspace(ops.make_norm_config(4, 128), device="cpu").numel() == 1256
