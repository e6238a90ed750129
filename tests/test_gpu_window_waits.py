"""The tcgen05 kernel of the windowed attention ends when its tiles stop getting done:
with a limit shorter than its run the call gives up, says so and leaves the layers
usable."""
import pytest
import torch

from test_gpu_tree_waits import DEV, _layer, kvc  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kmode,vmode,D", [("codebook", "int8", 128), ("uniform", "uniform", 64),
                                           ("uniform", "int8", 128), ("codebook", "uniform", 128)])
def test_wait_limit_times_out_and_recovers(kvc, kmode, vmode, D):  # noqa: F811
    """(Only that kernel can time out, so this also shows that it is the one that runs.)"""
    B, H, S = 2, 4, 30000
    gk, gv = _layer(kvc, kmode, B, H, D, S), _layer(kvc, vmode, B, H, D, S)
    q = torch.randn(B, H * 4, 100, D, generator=torch.Generator().manual_seed(9)).to(DEV)
    want = kvc.attend_window(gk, gv, q, 20000, 4)
    assert gk.sync_status() == 0 and bool(torch.isfinite(want).all())
    gk.set_wait_limit(1)
    for _ in range(3):
        kvc.attend_window(gk, gv, q, 20000, 4)
    assert gk.sync_status() == -5              # KVC_ETIMEOUT, read once
    assert gk.sync_status() == 0               # the error word was cleared
    gk.set_wait_limit(0)
    got = kvc.attend_window(gk, gv, q, 20000, 4)
    assert gk.sync_status() == 0 and torch.equal(got, want)
