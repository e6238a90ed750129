"""The tensor-core tree attention ends when its tiles stop getting done: with a
limit shorter than its run the call gives up, says so and leaves the layers
usable."""
import numpy as np
import pytest
import torch

from kvc_cases import fit_codebook

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rank_quantized_kv_gb300 as kvc

    kvc.load_library()
    return kvc


def _layer(kvc, mode, B, H, D, S):
    p = {}
    if mode == "codebook":
        p = fit_codebook(D, 3)
    elif mode == "uniform":
        p = dict(V=np.linalg.qr(np.random.default_rng(0).standard_normal((D, D)))[0][:, :48],
                 bits=np.full((1, 48), 4, np.uint8), qmin=np.full((1, 48), -3.0), qstep=np.full((1, 48), 0.4))
    lay = kvc.KVCacheLayer(mode, B, H, D, in_dtype="f16", capacity=S, device=DEV, **p)
    g = torch.Generator(device=DEV).manual_seed(5)
    for t in range(0, S, 8192):
        lay.append(torch.randn(B, H, min(8192, S - t), D, generator=g, device=DEV).half())
    return lay


@pytest.mark.parametrize("kmode,vmode,D,rep,N,S", [("codebook", "int8", 128, 2, 4, 250000),
                                                   ("uniform", "uniform", 64, 4, 8, 250000),
                                                   ("uniform", "int8", 128, 4, 15, 100000),
                                                   ("codebook", "uniform", 128, 8, 16, 100000)])
def test_wait_limit_times_out_and_recovers(kvc, kmode, vmode, D, rep, N, S):
    """16, 32, 64 and 128 columns.  (Only the tensor-core kernel can time out, so this
    also shows that it is the one that runs.)"""
    B, H = 2, 4
    gk, gv = _layer(kvc, kmode, B, H, D, S), _layer(kvc, vmode, B, H, D, S)
    q = torch.randn(B, H * rep, N, D, generator=torch.Generator().manual_seed(9)).to(DEV)
    want = kvc.attend_tree(gk, gv, q)
    assert gk.sync_status() == 0 and bool(torch.isfinite(want).all())
    gk.set_wait_limit(1)
    for _ in range(3):
        kvc.attend_tree(gk, gv, q)
    assert gk.sync_status() == -5              # KVC_ETIMEOUT, read once
    assert gk.sync_status() == 0               # the error word was cleared
    gk.set_wait_limit(0)
    got = kvc.attend_tree(gk, gv, q)
    assert gk.sync_status() == 0 and torch.equal(got, want)
