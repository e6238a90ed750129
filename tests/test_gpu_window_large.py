"""Windowed attention at sizes that keep the whole GPU busy, where jobs of 16, 32 and
128 rows take the place of those of eight: against the float64 oracle, within the
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

# rep, N, S of 4 slots: 12 rows, 24 rows, 600 rows of a slot
SIZES = {"16 rows": (4, 3, 20001), "32 rows": (8, 3, 10500), "128 rows": (4, 150, 1111)}


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rank_quantized_kv_gb300 as kvc

    kvc.load_library()
    return kvc


def _layers(kvc, kmode, vmode, D, S, bits=3, out="f16", seed=3, B=2, H=2):
    tree_cases.PATH[0] = "auto"
    return make_layers(kvc, kmode, vmode, B, H, D, S, seed, out=out, bits=bits, dev=DEV)


def _compare(kvc, layers, q, window, sinks, first=None, weights=False, decay=1.0, out=None, scale=0.0):
    gk, gv, rk, rv = layers
    B, H, S = gk.B, gk.H, len(gk)
    f = None if first is None else torch.tensor(first, dtype=torch.int32, device=DEV)
    w = w0 = None
    if weights:
        w0 = torch.rand(B, H, S, generator=torch.Generator().manual_seed(S))
        w = w0.to(DEV)
    o = kvc.attend_window(gk, gv, q.to(DEV), window, sinks, first=f, weights=w, decay=decay, out=out, scale=scale)
    torch.cuda.synchronize()
    assert gk.sync_status() == 0
    want, tol, ww, wtol = window_cases.reference(gk, rk, gv, rv, q.double().numpy(), scale or 1 / math.sqrt(gk.D),
                                                 window, sinks, first,
                                                 None if w0 is None else w0.double().numpy(), decay)
    window_cases.check(o, want, tol, "out")
    if weights:
        window_cases.check(w, ww, wtol, "weights")
    return o, w


def _q(rep, N, D, seed, dt="f32", B=2, H=2, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(B, H * rep, N, D, generator=g)).to(TORCH[dt])


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("kmode,vmode,bits,D", [("codebook", "int8", 3, 128), ("codebook", "uniform", 4, 128),
                                                ("codebook", "int8", 2, 64), ("uniform", "int8", 0, 128),
                                                ("uniform", "uniform", 0, 64), ("codebook", "int8", 1, 128)])
@pytest.mark.parametrize("window,sinks,weights", [(0, 0, False), (300, 5, True), (127, 200, False)])
def test_modes(kvc, size, kmode, vmode, bits, D, window, sinks, weights):
    rep, N, S = SIZES[size]
    _compare(kvc, _layers(kvc, kmode, vmode, D, S, bits), _q(rep, N, D, 1, "bf16"), window, sinks, weights=weights,
             decay=0.5)


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "uniform")])
@pytest.mark.parametrize("out", ["f16", "bf16"])
def test_padded_batch(kvc, size, kmode, vmode, out):
    """Padding that ends inside a tile, in the last tile, behind the last token; sinks
    behind it; queries that see nothing."""
    rep, N, S = SIZES[size]
    layers = _layers(kvc, kmode, vmode, 128, S, out=out)
    q = _q(rep, N, 128, 2, "f16")
    for first in ([0, 333], [S - 1, -7], [S - N // 2, 10 ** 8]):
        o, w = _compare(kvc, layers, q, 250, 9, first, weights=True, decay=0.0)
        if first[1] > S:
            assert bool((o[1] == 0).all()) and bool((w[1] == 0).all())


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("kmode", ["codebook", "uniform"])
@pytest.mark.parametrize("rising", [False, True])
def test_references_that_move(kvc, size, kmode, rising):
    """Scores and value scales that rise (or fall) over the cache by many times what
    the references allow before they move."""
    rep, N, S = SIZES[size]
    layers = _layers(kvc, kmode, "int8", 128, S)
    ramp = torch.logspace(-2, 1.2, S, device=DEV)
    if not rising:
        ramp = ramp.flip(0)
    for slot in range(4):
        for lay in layers[:2]:
            side = lay.slot_rows(slot)[1]
            if side is not None:
                h = side.view(torch.float16)[:, 0]
                h.copy_((h.float() * ramp).half())
    _compare(kvc, layers, _q(rep, N, 128, 3), 0, 0, weights=True)
    _compare(kvc, layers, _q(rep, N, 128, 3), 400, 3)


@pytest.mark.parametrize("size", list(SIZES))
def test_strided_arguments(kvc, size):
    """Output rows that start at any multiple of two bytes, transposed views."""
    rep, N, S = SIZES[size]
    layers = _layers(kvc, "codebook", "int8", 128, S)
    q = _q(rep, N, 128, 4, "bf16")
    plain, _ = _compare(kvc, layers, q, 500, 2)
    big = torch.full((2, N, 2 * rep, 131), 7.0, dtype=torch.float16, device=DEV)
    out = big[..., 1:129].transpose(1, 2)
    view = torch.empty(2, N, 2 * rep, 129, dtype=q.dtype, device=DEV)[..., 1:].transpose(1, 2)
    view.copy_(q)
    kvc.attend_window(layers[0], layers[1], view, 500, 2, out=out)
    assert torch.equal(out, plain)
    assert bool((big[..., 0] == 7).all()) and bool((big[..., 129:] == 7).all())


@pytest.mark.parametrize("size", list(SIZES))
def test_hidden_and_not_finite(kvc, size):
    """What hidden tokens hold has no effect; a visible norm or scale of NaN makes the
    rows that see it NaN, and only those."""
    rep, N, S = SIZES[size]
    gk, gv, rk, rv = _layers(kvc, "codebook", "int8", 128, S)
    q = _q(rep, N, 128, 5).to(DEV)
    first = torch.tensor([40, 0], dtype=torch.int32, device=DEV)
    kw = dict(window=64, sinks=8, first=first)
    a = kvc.attend_window(gk, gv, q, **kw)
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device=DEV).half()
    for slot in range(4):
        f = 40 if slot < 2 else 0
        hidden = torch.ones(S, dtype=torch.bool)
        hidden[f:f + 8] = False
        hidden[S - N - 64 + 1:] = False
        at = torch.nonzero(hidden).flatten().to(DEV)
        for lay in (gk, gv):
            lay.slot_rows(slot)[1].view(torch.float16)[at] = bad[torch.arange(len(at), device=DEV) % 3][:, None]
    assert torch.equal(a, kvc.attend_window(gk, gv, q, **kw))
    for lay in (gk, gv):
        side = lay.slot_rows(0)[1].view(torch.float16)
        keep = side[S - N].clone()
        side[S - N] = float("nan")  # seen by the queries 0 .. 63
        b = kvc.attend_window(gk, gv, q, **kw)
        assert bool(torch.isnan(b[0, :rep, :64]).all()) and torch.equal(b[0, :rep, 64:], a[0, :rep, 64:])
        assert torch.equal(b[0, rep:], a[0, rep:]) and torch.equal(b[1], a[1])
        side[S - N] = keep


@pytest.mark.parametrize("size", list(SIZES))
def test_repeats(kvc, size):
    """Equal bits from run to run."""
    rep, N, S = SIZES[size]
    gk, gv, rk, rv = _layers(kvc, "uniform", "int8", 128, S)
    q = _q(rep, N, 128, 6, "f16").to(DEV)
    got = []
    for _ in range(4):
        w = torch.zeros(2, 2, S, device=DEV)
        got.append((kvc.attend_window(gk, gv, q, 700, 4, weights=w), w))
    assert all(torch.equal(got[0][0], o) and torch.equal(got[0][1], w) for o, w in got)


def test_many_rows_over_few_tokens(kvc):
    """The weights' pass in shares of the rows: a prompt's queries over all of it."""
    layers = _layers(kvc, "uniform", "uniform", 64, 400, B=1, H=2)
    q = _q(8, 400, 64, 7, B=1)
    _compare(kvc, layers, q, 0, 0, weights=True, decay=0.25)
    _compare(kvc, layers, q, 50, 3, weights=True, decay=1.0)


@pytest.mark.parametrize("N", [1, 3, 40])
@pytest.mark.parametrize("what", ["keys", "values", "both"])
def test_rows_without_codes(kvc, N, what):
    """Layers whose components are all dropped: equal scores, or the mean alone."""
    rng = np.random.default_rng(0)
    B, H, D, S, rep = 2, 2, 64, 5000, 4

    def layer(empty, seed):
        r = 16
        V = np.linalg.qr(rng.standard_normal((D, D)))[0][:, :r].astype(np.float32)
        mean = rng.standard_normal(D).astype(np.float32)
        bits = np.full((1, r), 0 if empty else 4, np.uint8)
        lay = kvc.KVCacheLayer("uniform", B, H, D, V=V, mean=mean[None], bits=bits, qmin=np.full((1, r), -3.0),
                               qstep=np.full((1, r), 0.4), in_dtype="f16", capacity=S, device=DEV)
        lay.append(torch.randn(B, H, S, D, generator=torch.Generator().manual_seed(seed)).half().to(DEV))
        return lay

    gk, gv = layer(what != "values", 1), layer(what != "keys", 2)
    q = torch.randn(B, H * rep, N, D, generator=torch.Generator().manual_seed(3)).to(DEV)
    w = torch.zeros(B, H, S, device=DEV)
    o = kvc.attend_window(gk, gv, q, 4000, 2, weights=w).double()
    K, V = (lay.fetch().double() for lay in (gk, gv))
    pos, t = torch.arange(S - N, S, device=DEV)[:, None], torch.arange(S, device=DEV)
    seen = (t <= pos) & ((t > pos - 4000) | (t < 2))
    s = torch.einsum("bhrnd,bhsd->bhrns", q.double().view(B, H, rep, N, D), K) / D ** 0.5
    p = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
    want = torch.einsum("bhrns,bhsd->bhrnd", p, V).reshape(o.shape)
    # fetched rows are fp16: half a step of the largest each, and the output's own
    assert float((o - want).abs().max()) <= 4 * 2 ** -11 * float(V.abs().max())
    assert float((w - p.sum((2, 3))).abs().max()) <= 2e-3 * float(p.sum((2, 3)).max())
