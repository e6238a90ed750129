"""Windowed attention with finite scores so large that fp32 holds them to units or to
hundreds: every row is finite, and where one token stands out it is the output."""
import math

import numpy as np
import pytest
import torch

import tree_cases
from oracle.attend import window_visible
from tree_cases import make_layers, terms

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

# rep, N, S, window of 4 slots: jobs of 8, 16, 32 and 128 rows
SIZES = {"8 rows": (4, 2, 900, 0), "16 rows": (4, 3, 20001, 0), "32 rows": (8, 3, 14000, 0), "128 rows": (4, 150, 1111, 0)}
B, H, D = 2, 2, 128


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rank_quantized_kv_gb300 as kvc

    kvc.load_library()
    return kvc


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("kmode,path", [("codebook", "auto"), ("uniform", "auto"), ("codebook", "generic")])
@pytest.mark.parametrize("qscale", [2.0 ** 22, 2.0 ** 25, 2.0 ** 27, 2.0 ** 28, 2.0 ** 32])
@pytest.mark.parametrize("vscale", [1.0, 2.0 ** -9])
def test_scores_that_fp32_holds_coarsely(kvc, size, kmode, path, qscale, vscale):
    """A score is off by 2^-11 of the sum of its terms' magnitudes at most (centroids in
    fp16; all else is far less), twice for a difference: tokens that stay further than
    that and 64 behind the best one have weights of nothing."""
    rep, N, S, window = SIZES[size]
    tree_cases.PATH[0] = path
    gk, gv, rk, rv = make_layers(kvc, kmode, "int8", B, H, D, S, 47, dev=DEV)
    tree_cases.PATH[0] = "auto"
    for slot in range(B * H):
        gv.slot_rows(slot)[1].view(torch.float16).mul_(vscale)
    q = qscale * torch.randn(B, H * rep, N, D, generator=torch.Generator().manual_seed(S))
    o = kvc.attend_window(gk, gv, q.to(DEV), window)
    assert gk.sync_status() == 0 and bool(torch.isfinite(o).all())
    o = o.double().cpu().numpy()
    vis, scale, alone = window_visible(N, S, window), 1 / math.sqrt(D), 0
    for b in range(B):
        for h in range(H):
            K, TK, EK = terms(gk, rk, b * H + h)
            V, _, _ = terms(gv, rv, b * H + h)
            keys = np.abs(EK).T @ np.abs(TK).T
            for x in range(h * rep, (h + 1) * rep):
                qx = q[b, x].double().numpy()
                s = np.where(vis, scale * qx @ K.T, -np.inf)
                off = 2 * 2.0 ** -11 * scale * np.max(np.where(vis, np.abs(qx) @ keys, 0.0), axis=1) + 64
                best = np.argmax(s, axis=1)
                top = np.take_along_axis(s, best[:, None], 1)
                clear = ((s > top - off[:, None]).sum(1) == 1)
                alone += clear.sum()
                err = np.abs(o[b, x] - V[best])[clear]
                assert np.all(err <= 2.0 ** -10 * np.abs(V[best])[clear] + 2.0 ** -24)
    assert alone > 0
