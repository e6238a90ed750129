"""Tree attention with query rows that are not finite, or whose scores pass the
range of fp32: such a row's output is not finite either (zeros are for rows that
see no token), on both kernels, with any values and with caches in which no tile
of 128 tokens is wholly visible."""
import numpy as np
import pytest
import torch

import tree_cases
from tree_cases import make_layers, random_tree

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rank_quantized_kv_gb300 as kvc

    kvc.load_library()
    return kvc


@pytest.fixture(autouse=True, params=["auto", "generic"])
def path(request):
    tree_cases.PATH[0] = request.param
    yield
    tree_cases.PATH[0] = "auto"


@pytest.mark.parametrize("kmode", ["codebook", "uniform"])
@pytest.mark.parametrize("vmode", ["int8", "uniform"])
@pytest.mark.parametrize("S,first", [(84, 0), (84, 70), (84, 80), (300, 0), (300, 200), (5, 0)])
@pytest.mark.parametrize("rep,N", [(2, 4), (32, 4)])
def test_rows_of_nan_and_infinity(kvc, kmode, vmode, S, first, rep, N):
    B, H, D = 1, 1, 64
    gk, gv, _, _ = make_layers(kvc, kmode, vmode, B, H, D, S, 61, dev=DEV)
    mask = torch.from_numpy(random_tree(np.random.default_rng(S), B, N)).to(DEV)
    q = torch.randn(B, rep, N, D, generator=torch.Generator().manual_seed(7)).to(DEV)
    at = torch.tensor([first], dtype=torch.int32, device=DEV)
    good = kvc.attend_tree(gk, gv, q, mask=mask, first=at)
    assert bool(torch.isfinite(good).all())
    bad = [(0, 0, float("nan")), (0, 2, float("inf")), (1, 1, float("-inf")), (1, 3, float("nan"))]
    for x, i, v in bad:
        q[0, x, i] = v
    q[0, 0, 2, 3:] = 0.5  # infinities in some components alone
    o = kvc.attend_tree(gk, gv, q, mask=mask, first=at)
    for x in range(rep):
        for i in range(N):
            if any((x, i) == b[:2] for b in bad):
                assert not bool(torch.isfinite(o[0, x, i]).any()), (x, i)
            else:
                assert torch.equal(o[0, x, i], good[0, x, i]), (x, i)


@pytest.mark.parametrize("vmode", ["int8", "uniform"])
@pytest.mark.parametrize("S", [84, 700])
def test_scores_of_minus_infinity(kvc, vmode, S):
    """A row whose every visible score falls below fp32's range has no softmax: NaN.
    (Keys of dropped components: every token's score is q . mean.)  A row that sees
    nothing stays zero, the others stay what they were."""
    B, H, D, N = 1, 2, 64, 3
    rng = np.random.default_rng(0)
    mean = rng.standard_normal((H, D)).astype(np.float32)
    p = dict(V=1e-3 * rng.standard_normal((H, D, 4)), mean=mean, bits=np.zeros((H, 4), dtype=np.uint8),
             qmin=np.zeros((H, 4)), qstep=np.ones((H, 4)), basis_of=np.arange(H))
    gk = kvc.KVCacheLayer("uniform", B, H, D, in_dtype="f16", capacity=S, device=DEV,
                          path=tree_cases.PATH[0], **p)
    _, gv, _, _ = make_layers(kvc, "codebook", vmode, B, H, D, S, 62, dev=DEV)
    gk.append(torch.randn(B, H, S, D, device=DEV).half())
    q = torch.randn(B, H, N, D, generator=torch.Generator().manual_seed(7)).to(DEV)
    first = torch.tensor([S], dtype=torch.int32, device=DEV)
    mask = torch.tensor([[1, 0, 0], [1, 1, 0], [0, 0, 0]], dtype=torch.bool, device=DEV)
    for f in (None, first):
        q[0, 0, 1] = 0.25
        good = kvc.attend_tree(gk, gv, q, mask=mask, first=f)
        q[0, 0, 1] = torch.from_numpy(np.float32(-1e38) * np.sign(mean[0])).to(DEV)
        o = kvc.attend_tree(gk, gv, q, mask=mask, first=f)
        assert bool(torch.isnan(o[0, 0, 1]).all())
        assert torch.equal(o[0, 0, 0], good[0, 0, 0]) and torch.equal(o[0, 1], good[0, 1])
        assert torch.equal(o[0, 0, 2], good[0, 0, 2]) and bool(torch.isfinite(good).all())
        if f is not None:
            assert not bool(o[0, :, 2].any())


@pytest.mark.parametrize("S", [84, 300])
def test_nan_queries_over_values_of_dropped_components(kvc, S):
    """Values of which no component is kept are their mean whatever the weights
    are, but for a row whose weights are not numbers."""
    B, H, D, N = 1, 2, 64, 3
    gk, _, _, _ = make_layers(kvc, "codebook", "int8", B, H, D, S, 64, dev=DEV)
    rng = np.random.default_rng(1)
    mean = rng.standard_normal((H, D)).astype(np.float32)
    gv = kvc.KVCacheLayer("uniform", B, H, D, in_dtype="f16", capacity=S, device=DEV,
                          V=rng.standard_normal((H, D, 4)), mean=mean, bits=np.zeros((H, 4), dtype=np.uint8),
                          qmin=np.zeros((H, 4)), qstep=np.ones((H, 4)), basis_of=np.arange(H))
    gv.append(torch.randn(B, H, S, D, device=DEV).half())
    q = torch.randn(B, H, N, D, generator=torch.Generator().manual_seed(7)).to(DEV)
    q[0, 1, 1] = float("nan")
    o = kvc.attend_tree(gk, gv, q)
    want = torch.from_numpy(mean).to(DEV).half()
    assert bool(torch.isnan(o[0, 1, 1]).all())
    assert all(torch.equal(o[0, h, i], want[h]) for h in range(H) for i in range(N) if (h, i) != (1, 1))
