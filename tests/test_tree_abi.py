"""Tree attention, gather and accept without a GPU: calls that are refused
before anything touches a device, and the oracle's visibility."""
import ctypes

import numpy as np
import pytest

from oracle.attend import attend_rows, attend_tree_rows, tree_visible


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
    d = kvc._TreeDesc(Hq=1, N=1)
    assert lib.kvc_attend_tree_workspace_bytes(None, None, 1, 1, ctypes.byref(n)) == -2
    assert lib.kvc_attend_tree_workspace_bytes(None, None, 1, 1, None) == -1
    assert lib.kvc_attend_tree(None, None, ctypes.byref(d), None, 0, None) == -2
    assert lib.kvc_attend_tree(None, None, None, None, 0, None) == -1
    assert lib.kvc_gather(None, None, None, None, 0, 1, None) == -2
    assert lib.kvc_accept(None, 1, None, 1, None) == -2
    assert b"NULL" in lib.kvc_last_error()


def test_oracle_visibility():
    see = tree_visible(2, 5, first=1)
    assert see.astype(int).tolist() == [[0, 1, 1, 1, 0], [0, 1, 1, 1, 1]]
    see = tree_visible(2, 2, mask=[[0, 0], [1, 0]])
    assert see.astype(int).tolist() == [[0, 0], [1, 0]]
    assert not tree_visible(1, 4, first=9, mask=[[0]]).any()


def test_oracle_rows():
    """A draft equals a plain query over the tokens it sees; one that sees none is zero."""
    rng = np.random.default_rng(0)
    q, K, V = rng.standard_normal((3, 4)), rng.standard_normal((6, 4)), rng.standard_normal((6, 4))
    vis = tree_visible(3, 6, 1, [[1, 0, 0], [1, 1, 0], [0, 0, 1]])
    vis[2] = False
    out, p = attend_tree_rows(q, K, V, 0.5, vis)
    for i in (0, 1):
        t = np.flatnonzero(vis[i])
        assert np.allclose(out[i], attend_rows(q[i], K[t], V[t], 0.5), atol=1e-15)
        assert abs(p[i].sum() - 1) < 1e-15
    assert not out[2].any() and not p[2].any()
