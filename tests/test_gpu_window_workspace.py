"""The scratch of windowed attention: what it grows by, and that calls stay inside it."""
import pytest
import torch

import tree_cases
from tree_cases import make_layers

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
B, H, D = 2, 2, 128


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rank_quantized_kv_gb300 as kvc

    kvc.load_library()
    return kvc


def _layers(kvc, kmode, vmode, S):
    tree_cases.PATH[0] = "auto"
    return make_layers(kvc, kmode, vmode, B, H, D, S, 23, dev=DEV)[:2]


@pytest.mark.parametrize("kmode", ["codebook", "uniform"])
def test_bytes_of_a_prompts_row(kvc, kmode):
    """A row of many keeps its query in the keys' basis (two fp16 pieces of each of up to
    128 positions) and a few numbers; not a partial output, 512 bytes more, since jobs
    that lie in one CTA are written by it."""
    gk, gv = _layers(kvc, kmode, "int8", 4096)
    size = [kvc.attend_window_workspace_bytes(gk, gv, torch.empty(B, 8 * H, N, D, device=DEV), 1024)
            for N in (1024, 2048, 4096)]
    for n, a, b in ((1024, *size[:2]), (2048, *size[1:])):
        assert b - a <= B * H * 8 * n * (128 * 4 + 64)


@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "uniform"), ("uniform", "int8")])
@pytest.mark.parametrize("S,N,rep,window", [(900, 300, 3, 0), (2000, 1900, 2, 700), (1111, 150, 4, 520), (900, 2, 4, 0),
                                            (14000, 3, 8, 13600), (400, 400, 8, 0)])
@pytest.mark.parametrize("weights", [False, True])
def test_calls_stay_inside(kvc, kmode, vmode, S, N, rep, window, weights):
    """Cut jobs at every place of their runs: equal results whatever the scratch held
    before, and nothing behind its end is written."""
    gk, gv = _layers(kvc, kmode, vmode, S)
    q = torch.randn(B, H * rep, N, D, generator=torch.Generator().manual_seed(N)).to(DEV)
    w = torch.zeros(B, H, S, device=DEV) if weights else None
    want = kvc.attend_window(gk, gv, q, window, 5, weights=w)
    n = kvc.attend_window_workspace_bytes(gk, gv, q, window, 5, w)
    for fill in (0, 255):
        ws = torch.full((n + 4096,), fill, dtype=torch.uint8, device=DEV)
        x = None if w is None else torch.zeros_like(w)
        o = kvc.attend_window(gk, gv, q, window, 5, weights=x, workspace=ws[:n])
        assert torch.equal(o, want) and (w is None or torch.equal(w, x))
        assert bool((ws[n:] == fill).all())
