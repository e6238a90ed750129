"""GPU parity of windowed attention (kvc_attend_window) and of the weights that it
accumulates against the float64 oracle on the GPU's own stored rows, within the
allowance derived in window_cases.py."""
import math

import numpy as np
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


@pytest.fixture(autouse=True, params=["auto", "generic"])
def path(request):
    """Every test on the kernels that the layers' sizes choose and on those for any layer."""
    tree_cases.PATH[0] = request.param
    yield
    tree_cases.PATH[0] = "auto"


def _q(B, Hq, N, D, seed, dt="f32", scale=1.0):
    q = scale * torch.randn(B, Hq, N, D, generator=torch.Generator().manual_seed(seed))
    return q.to(TORCH[dt])


def _run(kvc, kmode, vmode, B, H, rep, D, S, N, window=0, sinks=0, first=None, dt="f32", out="f16", bits=3,
         weights=False, decay=1.0, qscale=1.0, scale=0.0, seed=None):
    """With and without weights, against the oracle; returns what was compared."""
    seed = seed if seed is not None else 1000 + S + 7 * N + D
    gk, gv, rk, rv = make_layers(kvc, kmode, vmode, B, H, D, S, seed, out=out, bits=bits, dev=DEV)
    q = _q(B, H * rep, N, D, seed, dt, qscale)
    f = None if first is None else torch.tensor(first, dtype=torch.int32, device=DEV)
    w = w0 = None
    if weights:
        w0 = torch.rand(B, H, S + 3, generator=torch.Generator().manual_seed(seed))
        w = w0.to(DEV)
    o = kvc.attend_window(gk, gv, q.to(DEV), window=window, sinks=sinks, first=f, scale=scale, weights=w,
                          decay=decay)
    torch.cuda.synchronize()
    assert gk.sync_status() == 0
    want, tol, ww, wtol = window_cases.reference(gk, rk, gv, rv, q.double().numpy(), scale or 1 / math.sqrt(D),
                                                 window, sinks, first,
                                                 None if w0 is None else w0.double().numpy(), decay)
    window_cases.check(o, want, tol, "out")
    if weights:
        window_cases.check(w[:, :, :S], ww, wtol, "weights")
        assert torch.equal(w[:, :, S:].cpu(), w0[:, :, S:]), "weights past the length were written"
    return gk, gv, q.to(DEV), f, o, w


@pytest.mark.parametrize("kmode,vmode,bits", [("codebook", "int8", 3), ("uniform", "uniform", 0),
                                              ("uniform", "int8", 0), ("codebook", "uniform", 4),
                                              ("codebook", "int8", 2), ("codebook", "int8", 8),
                                              ("codebook", "int8", 1), ("prod", "int8", 2),
                                              ("prod", "uniform", 2)])
@pytest.mark.parametrize("D,rep,N,S,window,sinks", [(128, 4, 1, 700, 200, 4), (64, 2, 5, 131, 0, 0),
                                                    (128, 3, 9, 300, 37, 70)])
@pytest.mark.parametrize("weights", [False, True])
def test_modes(kvc, kmode, vmode, bits, D, rep, N, S, window, sinks, weights):
    _run(kvc, kmode, vmode, 2, 2, rep, D, S, N, window, sinks, bits=bits, weights=weights)


@pytest.mark.parametrize("D", [20, 32, 96, 200, 256])
@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "uniform")])
def test_head_sizes(kvc, kmode, vmode, D):
    if kmode == "codebook" and D % 4:
        pytest.skip("3-bit rows of whole bytes are not needed here")
    _run(kvc, kmode, vmode, 1, 2, 3, D, 300, 4, 100, 3, weights=True)


@pytest.mark.parametrize("rep,N", [(1, 1), (1, 2), (3, 3), (8, 1), (8, 2), (5, 7), (4, 32), (16, 9), (1, 130),
                                   (7, 40)])
@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "uniform")])
def test_row_counts(kvc, kmode, vmode, rep, N):
    """Rows below, at and above one job's, over several tiles of tokens."""
    _run(kvc, kmode, vmode, 1, 2, rep, 128, 420, N, 90, 5, dt="bf16", weights=True)


@pytest.mark.parametrize("S,N", [(1, 1), (2, 2), (5, 5), (15, 1), (16, 1), (17, 3), (31, 2), (32, 32), (33, 1),
                                 (127, 3), (128, 128), (129, 3), (257, 130), (1025, 9), (4099, 1)])
@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "uniform")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 0), (33, 40), (10 ** 12, 10 ** 12)])
def test_lengths(kvc, kmode, vmode, S, N, window, sinks):
    """Lengths, windows and sinks at and around the tiles' ends, windows and sinks
    that meet, that overlap and that exceed the cache."""
    _run(kvc, kmode, vmode, 2, 1, 2, 64, S, N, window, sinks, dt="f16", weights=True, decay=0.0)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f16", "bf16"])
@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
def test_types(kvc, dt, out, decay):
    _run(kvc, "codebook", "int8", 1, 2, 2, 128, 300, 4, 64, 2, dt=dt, out=out, weights=True, decay=decay)
    _run(kvc, "uniform", "uniform", 1, 2, 2, 128, 300, 4, 64, 2, dt=dt, out=out, weights=True, decay=decay)


@pytest.mark.parametrize("N", [1, 6])
@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "uniform")])
def test_padded_batch(kvc, kmode, vmode, N):
    """Left padding from none to all tokens and beyond: rows that see nothing are
    zero whatever out held and give no weight; sinks count from the first token."""
    S = 700
    first = [0, -3, 150, 256, S - 1, 10 ** 6]
    gk, gv, q, f, o, w = _run(kvc, kmode, vmode, 6, 1, 4, 128, S, N, 100, 20, first, weights=True, decay=0.0)
    assert bool((o[5] == 0).all()) and bool((o[4, :, :N - 1] == 0).all()) and bool((w[5, :, :S] == 0).all())
    out = torch.full_like(o, float("nan"))
    kvc.attend_window(gk, gv, q, 100, 20, first=f, weights=torch.empty_like(w).fill_(float("nan")), decay=0.0,
                      out=out)
    assert torch.equal(out, o)


@pytest.mark.parametrize("scale,qscale", [(0.02, 1.0), (3.0, 1.0), (0.0, 1e-6), (1e-4, 3e3)])
@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "int8"), ("uniform", "uniform")])
def test_scales(kvc, kmode, vmode, scale, qscale):
    """From flat to peaked weights, tiny and large queries."""
    _run(kvc, kmode, vmode, 1, 2, 4, 128, 500, 2, 300, 4, scale=scale, qscale=qscale, weights=True)


def test_rows_of_zero_queries(kvc):
    """Scores all equal: the mean of the visible values, weights 1 / count."""
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", 1, 1, 128, 300, 5, dev=DEV)
    w = torch.zeros(1, 1, 300, device=DEV)
    kvc.attend_window(gk, gv, torch.zeros(1, 4, 1, 128, device=DEV), 64, 0, weights=w)
    want = torch.zeros(300)
    want[236:] = 4 / 64
    assert torch.equal(w[0, 0].cpu(), want)


@pytest.mark.parametrize("kmode", ["codebook", "prod"])
def test_hidden_tokens_hold_anything(kvc, kmode):
    """NaN and infinity in the norms and scales of tokens that no query sees."""
    B, H, rep, D, S, N = 2, 1, 4, 128, 600, 3
    gk, gv, rk, rv = make_layers(kvc, kmode, "int8", B, H, D, S, 17, dev=DEV)
    q = _q(B, H * rep, N, D, 3).to(DEV)
    first = torch.tensor([40, 0], dtype=torch.int32, device=DEV)
    w0 = torch.zeros(B, H, S, device=DEV)
    a = kvc.attend_window(gk, gv, q, 200, 8, first=first, weights=w0)
    seen = torch.zeros(B, S, dtype=torch.bool)
    for b, f in enumerate((40, 0)):
        seen[b, f:f + 8] = True
        seen[b, S - N - 200 + 1:] = True
    for slot in range(B):
        for lay in (gk, gv):
            side = lay.slot_rows(slot)[1].view(torch.float16)
            bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device=DEV).half()
            hidden = torch.nonzero(~seen[slot]).flatten().to(DEV)
            side[hidden] = bad[torch.arange(len(hidden), device=DEV) % 3][:, None]
    w1 = torch.zeros(B, H, S, device=DEV)
    b_ = kvc.attend_window(gk, gv, q, 200, 8, first=first, weights=w1)
    assert torch.equal(a, b_) and torch.equal(w0, w1)


def test_rows_that_are_not_finite(kvc):
    """A score of NaN or +inf makes the rows that see it NaN, and the weights of what they see."""
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", 1, 1, 128, 200, 21, dev=DEV)
    q = _q(1, 2, 2, 128, 4).to(DEV)
    gk.slot_rows(0)[1].view(torch.float16)[100] = float("nan")
    w = torch.zeros(1, 1, 200, device=DEV)
    o = kvc.attend_window(gk, gv, q, 99, 0, weights=w)  # query 0 sees 100 .. 198, query 1 101 .. 199
    assert bool(torch.isnan(o[0, :, 0]).all()) and bool(torch.isfinite(o[0, :, 1]).all())
    assert bool(torch.isnan(w[0, 0, 100:199]).all()) and bool((w[0, 0, :100] == 0).all())
    assert bool(torch.isfinite(w[0, 0, 199:]).all())
    q[0, 0, 1, 5] = float("inf")
    o = kvc.attend_window(gk, gv, q, 50, 0)
    assert bool(torch.isnan(o[0, 0, 1]).all()) and bool(torch.isfinite(o[0, 1]).all())


@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "uniform")])
def test_strided_arguments(kvc, kmode, vmode):
    """Queries, output and weights as views; what lies between their rows stays."""
    B, H, rep, D, S, N = 2, 2, 3, 128, 333, 5
    gk, gv, rk, rv = make_layers(kvc, kmode, vmode, B, H, D, S, 9, dev=DEV)
    q = _q(B, H * rep, N, D, 2, "bf16").to(DEV)
    w = torch.rand(B, H, S, device=DEV)
    plain = kvc.attend_window(gk, gv, q, 50, 3, weights=(wp := w.clone()))
    qv = torch.empty(B, N, H * rep, D + 8, dtype=q.dtype, device=DEV)[..., :D].transpose(1, 2)
    qv.copy_(q)
    big = torch.full((B, N, H * rep, D + 3), 7.0, dtype=torch.float16, device=DEV)
    wbig = torch.full((H, B, S + 9), 5.0, device=DEV)
    wv = wbig.transpose(0, 1)[:, :, 4:4 + S]
    wv.copy_(w)
    kvc.attend_window(gk, gv, qv, 50, 3, weights=wv, out=big[..., :D].transpose(1, 2))
    assert torch.equal(big[..., :D].transpose(1, 2), plain) and bool((big[..., D:] == 7).all())
    assert torch.equal(wv, wp) and bool((wbig[:, :, :4] == 5).all()) and bool((wbig[:, :, 4 + S:] == 5).all())


def test_shared_query(kvc):
    """Queries of stride 0: one vector for all heads and tokens."""
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", 1, 2, 128, 100, 9, dev=DEV)
    one = _q(1, 1, 1, 128, 2).to(DEV)
    a = kvc.attend_window(gk, gv, one.expand(1, 4, 3, 128), 20, 1)
    b = kvc.attend_window(gk, gv, one.expand(1, 4, 3, 128).contiguous(), 20, 1)
    assert torch.equal(a, b)


def test_agrees_with_the_other_attentions(kvc):
    """Without a window: a chain of drafts, and for one token plain decode attention."""
    gk, gv, rk, rv = make_layers(kvc, "uniform", "int8", 2, 2, 128, 400, 12, dev=DEV)
    q = _q(2, 8, 3, 128, 1).to(DEV)
    a, b = kvc.attend_window(gk, gv, q), kvc.attend_tree(gk, gv, q)
    assert float((a.float() - b.float()).abs().max()) <= 2 ** -9 * float(b.float().abs().max())
    a = kvc.attend_window(gk, gv, q[:, :, 2:])[:, :, 0]
    b = kvc.attend(gk, gv, q[:, :, 2].contiguous())
    assert float((a.float() - b.float()).abs().max()) <= 2 ** -9 * float(b.float().abs().max())


def test_repeats_and_streams(kvc):
    """Equal bits from run to run, from two streams at once and from a replayed graph."""
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", 4, 2, 128, 3000, 12, dev=DEV)
    q = _q(4, 8, 2, 128, 1, "f16").to(DEV)
    w = torch.zeros(4, 2, 3000, device=DEV)
    o = kvc.attend_window(gk, gv, q, 1000, 4, weights=w, decay=0.0)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s in side:
            x = torch.empty_like(w)
            with torch.cuda.stream(s):
                x.fill_(3.0)
            got.append((kvc.attend_window(gk, gv, q, 1000, 4, weights=x, decay=0.0, stream=s), x))
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) and torch.equal(w, x) for a, x in got)
    out, x = torch.empty_like(o), torch.empty_like(w)
    ws = torch.empty(kvc.attend_window_workspace_bytes(gk, gv, q, 1000, 4, x), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.attend_window(gk, gv, q, 1000, 4, weights=x, decay=0.0, out=out, workspace=ws)
    for _ in range(2):
        out.zero_()
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(x, w)


def test_long_cache(kvc):
    """A window behind 100000 tokens, sinks far away from it."""
    _run(kvc, "codebook", "int8", 1, 1, 2, 128, 100003, 2, 5000, 4, dt="f16", weights=True)


def test_refusals(kvc):
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", 2, 2, 128, 20, 3, dev=DEV)
    other, _, _, _ = make_layers(kvc, "codebook", "int8", 2, 2, 128, 19, 3, dev=DEV)
    q = _q(2, 4, 2, 128, 1).to(DEV)
    w = torch.zeros(2, 2, 20, device=DEV)

    def refused(k=gk, v=gv, q=q, **kw):
        with pytest.raises((kvc.KvcError, ValueError)):
            kvc.attend_window(k, v, q, **kw)

    refused(window=-1)
    refused(sinks=-1)
    refused(v=gk)
    refused(k=other)
    refused(q=q[:, :3])
    refused(q=torch.zeros(2, 4, 21, 128, device=DEV))
    refused(q=torch.zeros(2, 4, 0, 128, device=DEV))
    refused(q=q.cpu())
    refused(scale=-1.0)
    refused(scale=float("nan"))
    refused(weights=w, decay=-0.5)
    refused(weights=w, decay=float("inf"))
    refused(weights=w.cpu())
    refused(weights=w[:, :, :19])
    refused(weights=torch.zeros(2, 1, 20, device=DEV).expand(2, 2, 20))
    refused(out=torch.empty(2, 1, 2, 128, dtype=torch.float16, device=DEV).expand(2, 4, 2, 128))
    refused(out=torch.empty(2, 4, 2, 128, device=DEV))
    refused(first=torch.zeros(2, dtype=torch.int32))
    refused(workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert gk.sync_status() == 0
    kvc.attend_window(gk, gv, q, weights=w)  # and the layers still work
