"""The two softmax groups of the windowed attention's kernel for many rows: jobs of one
tile of 128 tokens, where a group has none and reads the other's sums, of two and of
odd counts, cut between CTAs and whole, one after another in a CTA."""
import math

import pytest
import torch

import tree_cases
import window_cases
from tree_cases import TORCH, make_layers

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rank_quantized_kv_gb300 as kvc

    kvc.load_library()
    return kvc


@pytest.mark.parametrize("kmode", ["codebook", "uniform"])
@pytest.mark.parametrize("B,S,N,window", [(20, 128, 32, 0), (20, 127, 40, 90), (22, 256, 32, 0), (24, 300, 33, 140),
                                          (24, 384, 128, 0)])
def test_groups_with_few_tiles(kvc, kmode, B, S, N, window):
    """(80 and more slots of 128 and more rows: past the sizes that take jobs of eight rows.)"""
    tree_cases.PATH[0] = "auto"
    H, rep, D = 4, 4, 64
    gk, gv, rk, rv = make_layers(kvc, kmode, "int8", B, H, D, S, 31, dev=DEV)
    q = torch.randn(B, H * rep, N, D, generator=torch.Generator().manual_seed(S)).to(TORCH["bf16"])
    o = kvc.attend_window(gk, gv, q.to(DEV), window, 3)
    for _ in range(5):
        assert torch.equal(o, kvc.attend_window(gk, gv, q.to(DEV), window, 3))
    assert gk.sync_status() == 0
    want, tol, _, _ = window_cases.reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(D), window, 3)
    window_cases.check(o, want, tol, "out")
