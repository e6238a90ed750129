"""Windowed attention and eviction without a GPU: calls that are refused before
anything touches a device, and the oracle's visibility and choice."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.attend import evicted, window_visible


@pytest.fixture(scope="module")
def kvc():
    import rank_quantized_kv_gb300 as kvc

    try:
        kvc.load_library()
    except ImportError:
        import __graft_entry__

        __graft_entry__.build()
        kvc.load_library()
    return kvc


def test_null_layers_and_descriptors(kvc):
    lib = kvc.load_library()
    n = ctypes.c_size_t()
    d = kvc._WindowDesc(Hq=1, N=1)
    assert lib.kvc_attend_window_workspace_bytes(None, None, ctypes.byref(d), ctypes.byref(n)) == -2
    assert lib.kvc_attend_window_workspace_bytes(None, None, ctypes.byref(d), None) == -1
    assert lib.kvc_attend_window(None, None, ctypes.byref(d), None, 0, None) == -2
    e = kvc._EvictDesc(keep=1)
    assert lib.kvc_evict(None, None, ctypes.byref(e), None) == -2
    assert b"NULL" in lib.kvc_last_error()


class _Layer:
    """The attributes that the binding's own checks look at."""
    B, H, D, device, _h, _lib = 2, 3, 8, "cpu", None, None

    def __len__(self):
        return 5


def test_binding_checks(kvc):
    lay = _Layer()
    q = torch.zeros(2, 6, 1, 8)
    for bad in (q[:1], q[0], q.double(), q.transpose(2, 3), torch.zeros(2, 6, 1, 4)):
        with pytest.raises(ValueError):
            kvc._window_desc(lay, lay, bad, 0, 0, None, 0.0, None, 1.0)
    for first in (torch.zeros(3, dtype=torch.int32), torch.zeros(2), torch.zeros(4, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            kvc._window_desc(lay, lay, q, 0, 0, first, 0.0, None, 1.0)
        with pytest.raises(ValueError):
            kvc.evict(lay, lay, None, 1, first=first)
    for w in (torch.zeros(2, 3, 4), torch.zeros(2, 3, 5, dtype=torch.float64), torch.zeros(3, 2, 5),
              torch.zeros(2, 3, 10)[:, :, ::2], torch.zeros(2, 15)):
        with pytest.raises(ValueError):
            kvc._window_desc(lay, lay, q, 0, 0, None, 0.0, w, 1.0)
        with pytest.raises(ValueError):
            kvc.evict(lay, lay, w, 1)
    d = kvc._window_desc(lay, lay, q, None, 4, None, 0.0, torch.zeros(2, 3, 7), 1.0)
    assert (d.window, d.sinks, d.weights_stride_b, d.weights_stride_h, d.N, d.Hq) == (0, 4, 21, 7, 1, 6)


def test_oracle_visibility():
    see = window_visible(2, 6, window=2, sinks=1, first=1)
    assert see.astype(int).tolist() == [[0, 1, 0, 1, 1, 0], [0, 1, 0, 0, 1, 1]]
    assert window_visible(1, 4).all() and not window_visible(1, 4, 2, 9, first=4).any()
    assert window_visible(2, 4, window=1, sinks=0, first=-5).astype(int).tolist() == [[0, 0, 1, 0], [0, 0, 0, 1]]


def test_oracle_choice():
    w = [5.0, 1.0, 1.0, 9.0, float("nan"), 0.0, -0.0, 2.0]
    assert evicted(w, 3).tolist() == [0, 3, 7]
    assert evicted(w, 4).tolist() == [0, 1, 3, 7]          # the earlier of two equals
    assert evicted(w, 6).tolist() == [0, 1, 2, 3, 5, 7]    # 0 and -0 are equal
    assert evicted(w, 3, sinks=1, recent=2).tolist() == [0, 6, 7]
    assert evicted(w, 7).tolist() == [0, 1, 2, 3, 5, 6, 7]  # NaN is the first to go
    assert evicted(w, 3, sinks=1, first=4).tolist() == [4, 5, 7]
    assert evicted(w, 6, first=4).tolist() == [0, 1, 4, 5, 6, 7]
    assert evicted(5, 2, recent=1).tolist() == [0, 4]
