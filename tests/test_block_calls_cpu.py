"""What the block operators' entry points refuse and which device they ask,
on the CPU: nothing here reaches a device."""
import ctypes
import types

import pytest
import torch

from matrix_aware_optimizer_gb300 import blocks, build, native as N

from .test_blocks_cpu import _desc


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return N.load()


@pytest.mark.parametrize("rows,d", [(1 << 31, 257), ((1 << 32) - 1, 8192), (1 << 32, 1)])
def test_norm_calls_agree_on_their_most_rows(lib, rows, d):
    desc, n = _desc(rows=rows, rows_per_sample=rows, d=d), ctypes.c_size_t()
    assert lib.prm_block_norm_forward(desc, 16, 16, 16, 16, 16, None) == N.PRM_ERR_UNSUPPORTED
    assert lib.prm_block_norm_workspace(desc, n) == N.PRM_ERR_UNSUPPORTED
    assert lib.prm_block_norm_backward(desc, 16, 16, 16, 16, 16, 16, 16, None, None, None, None, None, None, 0,
                                       None) == N.PRM_ERR_UNSUPPORTED


@pytest.mark.parametrize("rows,d", [((1 << 31) - 1, 8192), ((1 << 32) - 1, 256)])
def test_norm_takes_the_rows_below(lib, rows, d):
    n = ctypes.c_size_t()
    assert lib.prm_block_norm_workspace(_desc(rows=rows, rows_per_sample=rows, d=d, pre_weight=16), n) == N.PRM_OK


# -------------------------------------------------------------------- devices
class _Devices:
    """Stands in for torch.cuda's notion of the current device."""

    def __init__(self, monkeypatch):
        self.current, outer = 0, self

        class device:
            def __init__(self, d):
                self.index = d if isinstance(d, int) else d.index

            def __enter__(self):
                self.before, outer.current = outer.current, self.index

            def __exit__(self, *_):
                outer.current = self.before

        monkeypatch.setattr(torch.cuda, "device", device)


def _stream(index):
    return types.SimpleNamespace(device=torch.device("cuda", index), cuda_stream=77)


def test_status_is_read_on_the_streams_device(monkeypatch):
    devices, asked = _Devices(monkeypatch), []

    def status(stream):
        asked.append((devices.current, stream))
        return N.PRM_OK

    monkeypatch.setattr(N, "load", lambda: types.SimpleNamespace(prm_blocks_sync_status=status))
    blocks.blocks_sync_status(_stream(1))
    blocks.blocks_sync_status(_stream(0))
    assert asked == [(1, 77), (0, 77)] and devices.current == 0


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(blocks, "_current_device", lambda: 0)
    with pytest.raises(ValueError):
        blocks._is_elsewhere(0, _stream(1))
    with pytest.raises(ValueError):
        blocks._is_elsewhere(1, _stream(0))
    assert blocks._is_elsewhere(1, _stream(1)) and blocks._is_elsewhere(0, _stream(0))
    assert blocks._is_elsewhere(1, None) and not blocks._is_elsewhere(0, None)
