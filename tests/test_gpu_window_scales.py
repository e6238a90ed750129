"""Windowed attention over value scales that differ by many orders of magnitude: what a
query does not see has no effect on its row, whether no query sees it or others of the
same call do, and a row is as exact as its own visible tokens allow.

Allowance of a row: as in window_cases.py, but for the weights below fp16's normal
range.  A weight times a value scale is held to 2^-25 (half a step of fp16's smallest
numbers) of a unit by which the row's largest weight is 2^4 at least and the largest
scale that it sees 2^-1 at least: S tokens add at most S 2^-25 / (2^4 2^-1) = S 2^-28 of
the largest visible value."""
import math

import numpy as np
import pytest
import torch

import tree_cases
from oracle.attend import attend_tree_rows, window_visible
from tree_cases import TORCH, make_layers, terms
from window_cases import OUT_EPS, check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

# rep, N, S, window of 4 slots: jobs of 8, 16, 32 and 128 rows (longer calls of more rows
# take the larger jobs)
SIZES = {"8 rows": (4, 2, 900, 100), "16 rows": (4, 3, 20001, 19800), "32 rows": (8, 3, 14000, 13600),
         "128 rows": (4, 150, 1111, 520)}
B, H, D = 2, 2, 128
SINKS = 8


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rank_quantized_kv_gb300 as kvc

    kvc.load_library()
    return kvc


def _case(kvc, size, kmode, dt="bf16", path="auto"):
    rep, N, S, window = SIZES[size]
    tree_cases.PATH[0] = path
    layers = make_layers(kvc, kmode, "int8", B, H, D, S, 41, dev=DEV)
    tree_cases.PATH[0] = "auto"
    q = torch.randn(B, H * rep, N, D, generator=torch.Generator().manual_seed(S)).to(TORCH[dt])
    return layers, q, rep, N, S, window


def _scales(gv, slot):
    return gv.slot_rows(slot)[1].view(torch.float16)[:, 0]


def _run(kvc, layers, q, window, weights=False, **kw):
    w = torch.zeros(B, H, len(layers[0]), device=DEV) if weights else None
    o = kvc.attend_window(layers[0], layers[1], q.to(DEV), window, SINKS, weights=w, **kw)
    assert layers[0].sync_status() == 0
    return o, w


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("kmode,weights", [("codebook", False), ("uniform", False), ("uniform", True)])
@pytest.mark.parametrize("value", [65504.0, 3.0])
def test_scales_that_no_query_sees(kvc, size, kmode, weights, value):
    """Padding, what lies between the sinks and the window, in tiles of visible tokens
    and others."""
    layers, q, rep, N, S, window = _case(kvc, size, kmode)
    first = (40, 0)
    kw = dict(weights=weights, first=torch.tensor(first, dtype=torch.int32, device=DEV))
    for slot in range(B * H):  # small ones beside them
        _scales(layers[1], slot).mul_(0.05)
    a, wa = _run(kvc, layers, q, window, **kw)
    for slot in range(B * H):
        hidden = torch.ones(S, dtype=torch.bool, device=DEV)
        hidden[first[slot // H]:first[slot // H] + SINKS] = False
        hidden[S - N - window + 1:] = False
        _scales(layers[1], slot)[hidden] = value
    b, wb = _run(kvc, layers, q, window, **kw)
    assert torch.equal(a, b)
    assert not weights or torch.equal(wa, wb)


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("kmode", ["codebook", "uniform"])
@pytest.mark.parametrize("value", [65504.0, float("inf"), float("nan")])
def test_scales_that_other_queries_see(kvc, size, kmode, value):
    """The last token belongs to the last query alone, the first one of the first query's
    window to that query alone: the rows of the others are the same to the bit."""
    layers, q, rep, N, S, window = _case(kvc, size, kmode)
    for slot in range(B * H):
        _scales(layers[1], slot).mul_(0.05)
    a, _ = _run(kvc, layers, q, window)
    for slot in range(B * H):
        _scales(layers[1], slot)[S - 1] = value
    b, _ = _run(kvc, layers, q, window)
    assert torch.equal(a[:, :, :N - 1], b[:, :, :N - 1])
    assert not torch.equal(a[:, :, N - 1], b[:, :, N - 1])
    for slot in range(B * H):
        _scales(layers[1], slot)[S - N - window + 1] = value
    c, _ = _run(kvc, layers, q, window)
    assert torch.equal(b[:, :, 1:N - 1], c[:, :, 1:N - 1])
    assert not torch.equal(a[:, :, 0], c[:, :, 0])


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("kmode", ["codebook", "uniform"])
@pytest.mark.parametrize("pattern", ["first row", "last row", "falling", "rising", "a few"])
def test_rows_are_as_exact_as_what_they_see(kvc, size, kmode, pattern):
    """Against float64.  Scales that differ by up to 2^20 between tokens."""
    layers, q, rep, N, S, window = _case(kvc, size, kmode, "f32")
    gk, gv, rk, rv = layers
    for slot in range(B * H):
        s = _scales(gv, slot)
        if pattern == "first row":
            s[S - N - window + 1] = 6e4
        elif pattern == "last row":
            s[S - 1] = 6e4
        elif pattern == "a few":
            s[torch.arange(5, S, 37, device=DEV)] *= 300.0
        else:
            ramp = torch.logspace(-3, 3, window + N, device=DEV)
            s[S - window - N:] *= ramp if pattern == "rising" else ramp.flip(0)
    o, _ = _run(kvc, layers, q, window)
    want, tol = np.zeros(q.shape), np.zeros(q.shape)
    scale, eps = 1 / math.sqrt(D), 2.0 ** -15 + (2.0 ** -11 if kmode == "codebook" else 0.0)
    vis = window_visible(N, S, window, SINKS)
    for b in range(B):
        for h in range(H):
            K, TK, EK = terms(gk, rk, b * H + h)
            V, TV, EV = terms(gv, rv, b * H + h)
            av, keys = np.abs(TV), np.abs(EK).T @ np.abs(TK).T
            most = np.stack([av[v].max(0) for v in vis]) @ np.abs(EV)
            for x in range(h * rep, (h + 1) * rep):
                qx = q[b, x].double().numpy()
                r, p = attend_tree_rows(qx, K, V, scale, vis)
                delta = eps * scale * np.max(np.where(vis, np.abs(qx) @ keys, 0.0), axis=1)
                terms_v = (p @ av) @ np.abs(EV)
                want[b, x] = r
                tol[b, x] = (OUT_EPS["f16"] * np.abs(r) + (2.0 ** -11 + 2 * delta[:, None] + 2.0 ** -18) * terms_v
                             + S * 2.0 ** -28 * most + 2.0 ** -18 * (np.abs(r) + terms_v) + 2.0 ** -25)
    fits = np.abs(want) < 65000.0  # (a value past fp16's range is an infinity)
    assert fits.mean() > 0.5
    check(torch.where(torch.from_numpy(fits).to(DEV), o, torch.zeros_like(o)), np.where(fits, want, 0.0), tol, pattern)


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("kmode,vmode,path", [("codebook", "int8", "auto"), ("uniform", "uniform", "auto"),
                                              ("prod", "int8", "auto"), ("codebook", "int8", "generic")])
def test_later_queries_tokens_hold_anything(kvc, size, kmode, vmode, path):
    """Codes, norms and scales of the last token, which the last query alone sees."""
    rep, N, S, window = SIZES[size]
    tree_cases.PATH[0] = path
    gk, gv, _, _ = make_layers(kvc, kmode, vmode, B, H, D, S, 43, dev=DEV)
    tree_cases.PATH[0] = "auto"
    q = torch.randn(B, H * rep, N, D, generator=torch.Generator().manual_seed(S)).to(DEV)
    a = kvc.attend_window(gk, gv, q, window, SINKS)
    for lay in (gk, gv):
        for slot in range(B * H):
            rows, side = lay.slot_rows(slot)
            rows[S - 1] = 0xA7
            if side is not None:
                side[S - 1].view(torch.float16).fill_(float("inf") if slot % 2 else float("nan"))
    b = kvc.attend_window(gk, gv, q, window, SINKS)
    assert torch.equal(a[:, :, :N - 1], b[:, :, :N - 1])


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("kmode,path", [("uniform", "auto"), ("codebook", "auto"), ("codebook", "generic")])
@pytest.mark.parametrize("at", ["last token", "a token that all see", "a sink", "tokens around a tile's end"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_weights_do_not_depend_on_the_values(kvc, size, kmode, path, at, value):
    """A value scale of NaN makes the rows that see it NaN, one of infinity not finite;
    the weights stay what they are."""
    layers, q, rep, N, S, window = _case(kvc, size, kmode, path=path)
    a, wa = _run(kvc, layers, q, window, weights=True)
    tokens = {"last token": [S - 1], "a token that all see": [S - N - 7], "a sink": [SINKS - 1],
              "tokens around a tile's end": [S // 128 * 128 - 1, S // 128 * 128]}[at]
    for slot in range(B * H):
        _scales(layers[1], slot)[tokens] = value
    b, wb = _run(kvc, layers, q, window, weights=True)
    assert bool(torch.isfinite(wa).all()) and torch.equal(wa, wb)
    seen = torch.from_numpy(window_visible(N, S, window, SINKS))[:, tokens].any(1)
    assert torch.equal(a[:, :, ~seen], b[:, :, ~seen])
    hit = b[:, :, seen]
    if value != value:
        assert bool(torch.isnan(hit).all())
    else:
        assert not bool(torch.isfinite(hit).all(-1).any())
