"""GPU tests of eviction (kvc_evict): the chosen tokens and the moved rows are equal
to the oracle's choice and to the rows as they were, byte for byte."""
import numpy as np
import pytest
import torch

import window_cases
from oracle.attend import evicted
from tree_cases import make_layers

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rank_quantized_kv_gb300 as kvc

    kvc.load_library()
    return kvc


def _rows(lay):
    got = []
    for s in range(lay.n_slots):
        r, side = lay.slot_rows(s)
        got.append((r.clone(), None if side is None else side.clone()))
    return got


def _weights(B, H, S, seed, kind="random"):
    rng = np.random.default_rng(seed)
    w = np.exp(2 * rng.standard_normal((B, H, S))).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 3, (B, H, S)).astype(np.float32)
        w[rng.random(w.shape) < 0.2] = -0.0
    elif kind == "odd":
        for v in (np.nan, np.inf, -np.inf, -1.0, -0.0, 0.0, 1e-45, -1e-45, 3e38):
            w[rng.random(w.shape) < 0.08] = v
    elif kind == "equal":
        w[:] = 0.25
    return w


def _empty_twin(kvc, lay, params, cap):
    return kvc.KVCacheLayer(lay.mode, lay.B, lay.H, lay.D, in_dtype="f16", out_dtype=lay.out_dtype,
                            capacity=cap, device=DEV, **params)


def _check(index, rows, lay, before, want, base=0):
    B, H = lay.B, lay.H
    assert index.dtype == torch.int32 and index.shape == (B, H, want.shape[-1])
    assert np.array_equal(index.cpu().numpy(), want)
    after = _rows(lay)
    n = want.shape[-1]
    for s in range(B * H):
        at = torch.from_numpy(want.reshape(B * H, n)[s]).to(DEV)
        for was, now in zip(before[s], after[s]):
            if was is not None:
                assert torch.equal(now[base:base + n], was[at]), f"slot {s}"


def _run(kvc, kmode, vmode, B, H, D, S, keep, sinks=0, recent=0, first=None, kind="random", place="same", seed=0,
         weights=True, bits=3):
    gk, gv, rk, rv = make_layers(kvc, kmode, vmode, B, H, D, S, 50 + seed, bits=bits, dev=DEV, capacity=S + 5)
    w = _weights(B, H, S, seed, kind)
    want = np.stack([[evicted(w[b, h] if weights else S, keep, sinks, recent, 0 if first is None else first[b])
                      for h in range(H)] for b in range(B)])
    room = torch.full((B, H, S + 7), -5.0, device=DEV)
    wd = room[:, :, 2:2 + S]  # starts 8 bytes into a row
    wd.copy_(torch.from_numpy(w))
    f = None if first is None else torch.tensor(first, dtype=torch.int32, device=DEV)
    bk, bv = _rows(gk), _rows(gv)
    kept = torch.gather(wd, 2, torch.from_numpy(want).to(DEV))
    if place == "same":
        index, fo = kvc.evict(gk, gv, wd if weights else None, keep, sinks, recent, first=f)
        dk, dv, base = gk, gv, 0
        assert len(gk) == len(gv) == keep
        if weights:
            assert torch.equal(wd[:, :, :keep].nan_to_num(-77), kept.nan_to_num(-77))
            assert bool((wd[:, :, keep:] == 0).all())
            assert bool((room[:, :, :2] == -5).all()) and bool((room[:, :, 2 + S:] == -5).all())
    else:
        base = 3
        dk, dv, _, _ = make_layers(kvc, kmode, vmode, B, H, D, S, 50 + seed, bits=bits, dev=DEV, capacity=S + 5)
        dk.trim(S - min(base, S)), dv.trim(S - min(base, S))
        base = len(dk)
        head = _rows(dk)
        dw = torch.full((B, H, base + keep + 2), -5.0, device=DEV)
        index, fo = kvc.evict(gk, gv, wd if weights else None, keep, sinks, recent, first=f, into=(dk, dv, dw))
        assert len(dk) == len(dv) == base + keep and len(gk) == S
        got = dw[:, :, base:base + keep]
        assert torch.equal(got.nan_to_num(-77), (kept if weights else torch.zeros_like(got)).nan_to_num(-77))
        assert bool((dw[:, :, :base] == -5).all()) and bool((dw[:, :, base + keep:] == -5).all())
        for s in range(B * H):
            assert torch.equal(dk.slot_rows(s)[0][:base], head[s][0])
            assert torch.equal(gk.slot_rows(s)[0], bk[s][0])
    torch.cuda.synchronize()
    _check(index, None, dk, bk, want, base)
    _check(index, None, dv, bv, want, base)
    if first is None:
        assert fo is None
    else:
        assert fo.tolist() == [max(0, keep - (S - min(max(x, 0), S))) for x in first]
    assert dk.sync_status() == 0 and dv.sync_status() == 0
    return gk, gv


@pytest.mark.parametrize("place", ["same", "into"])
@pytest.mark.parametrize("kmode,vmode,bits", [("codebook", "int8", 3), ("uniform", "uniform", 0),
                                              ("codebook", "uniform", 1), ("prod", "int8", 2)])
@pytest.mark.parametrize("D,S,keep,sinks,recent", [(128, 700, 300, 4, 32), (64, 131, 130, 0, 0), (32, 57, 1, 0, 0),
                                                   (128, 40, 40, 7, 9)])
def test_modes(kvc, place, kmode, vmode, bits, D, S, keep, sinks, recent):
    _run(kvc, kmode, vmode, 2, 3, D, S, keep, sinks, recent, place=place, bits=bits)


@pytest.mark.parametrize("place", ["same", "into"])
@pytest.mark.parametrize("kind", ["random", "ties", "odd", "equal"])
@pytest.mark.parametrize("S,keep,sinks,recent", [(1, 1, 0, 0), (2, 1, 0, 1), (2047, 1000, 1, 1), (2049, 2048, 0, 0),
                                                 (5000, 77, 0, 76), (9000, 4000, 64, 300), (33000, 32000, 4, 0)])
def test_choice(kvc, place, kind, S, keep, sinks, recent):
    """Weights with ties, NaN, infinities and zeros of both signs, at and around the
    steps of the selection, with one and several blocks for a slot."""
    _run(kvc, "codebook", "int8", 1, 2, 64, S, keep, sinks, recent, kind=kind, place=place, seed=S)


@pytest.mark.parametrize("place", ["same", "into"])
@pytest.mark.parametrize("keep,sinks,recent", [(300, 5, 20), (20, 15, 5), (699, 0, 0), (1, 1, 0)])
def test_padded_batch(kvc, place, keep, sinks, recent):
    """Padding goes first and what is left of it stays in front; more padding than
    tokens kept, all tokens padding."""
    _run(kvc, "uniform", "int8", 6, 1, 64, 700, keep, sinks, recent, first=[0, -4, 10, 350, 699, 10 ** 6],
         place=place, kind="ties")


@pytest.mark.parametrize("place", ["same", "into"])
def test_without_weights(kvc, place):
    """Sinks and the most recent alone: a streaming cache; the rest goes to the earliest."""
    _run(kvc, "codebook", "int8", 2, 2, 128, 500, 104, 4, 100, weights=False, place=place)
    _run(kvc, "codebook", "int8", 2, 2, 128, 500, 110, 4, 100, weights=False, place=place)


def test_long_cache(kvc):
    """Several rounds of every cluster, rows of 48 and 128 bytes, in place."""
    _run(kvc, "codebook", "int8", 1, 2, 128, 70001, 60007, 4, 1000, kind="ties")


def test_many_slots(kvc):
    _run(kvc, "codebook", "int8", 16, 20, 32, 100, 63, 1, 5, place="same")
    _run(kvc, "codebook", "int8", 16, 20, 32, 100, 63, 1, 5, place="into")


def test_repeated_and_captured(kvc):
    """The same bits from run to run, and from a graph that evicts into other layers."""
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", 2, 2, 128, 3000, 4, dev=DEV)
    dk, dv, _, _ = make_layers(kvc, "codebook", "int8", 2, 2, 128, 3000, 4, dev=DEV)
    w = torch.from_numpy(_weights(2, 2, 3000, 1)).to(DEV)
    dw = torch.zeros(2, 2, 1000, device=DEV)
    dk.trim(3000), dv.trim(3000)
    index, _ = kvc.evict(gk, gv, w, 1000, 4, 100, into=(dk, dv, dw))
    rows, kept = _rows(dk), dw.clone()
    g = torch.cuda.CUDAGraph()
    dk.trim(1000), dv.trim(1000)
    with torch.cuda.graph(g):
        index2, _ = kvc.evict(gk, gv, w, 1000, 4, 100, into=(dk, dv, dw))
    for _ in range(2):
        for lay in (dk, dv):
            for s in range(4):
                lay.slot_rows(s)[0].zero_()
        dw.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(index, index2) and torch.equal(dw, kept)
        assert all(torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) for a, b in zip(rows, _rows(dk)))


def test_refusals(kvc):
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", 2, 2, 128, 20, 3, dev=DEV)
    dk, dv, _, _ = make_layers(kvc, "codebook", "int8", 2, 2, 128, 20, 3, dev=DEV)
    odd, _, _, _ = make_layers(kvc, "codebook", "int8", 2, 2, 128, 19, 3, dev=DEV)
    unlike, _, _, _ = make_layers(kvc, "codebook", "int8", 2, 2, 128, 4, 3, bits=2, dev=DEV)
    w = torch.rand(2, 2, 20, device=DEV)

    def refused(k=gk, v=gv, w=w, keep=10, **kw):
        with pytest.raises((kvc.KvcError, ValueError)):
            kvc.evict(k, v, w, keep, **kw)

    refused(keep=0)
    refused(keep=-1)
    refused(keep=21)
    refused(sinks=-1)
    refused(sinks=6, recent=5)
    refused(sinks=2 ** 62, recent=2 ** 62)
    refused(k=odd)
    refused(v=gk)
    refused(w=w.cpu())
    refused(w=w[:, :, :19])
    refused(w=torch.rand(2, 1, 20, device=DEV).expand(2, 2, 20))
    refused(into=(gk, gv, None))
    refused(into=(dk, dv, None))  # full
    dk.trim(20)
    refused(into=(dk, dv, None))  # of different lengths
    dv.trim(20)
    refused(into=(unlike, dv, None))
    refused(into=(dk, dv, torch.zeros(2, 2, 9, device=DEV)))
    refused(into=(dk, dv, w))
    refused(first=torch.zeros(2, dtype=torch.int32))
    assert len(gk) == 20 and len(dk) == 0
    kvc.evict(gk, gv, w, 10, into=(dk, dv, None))  # and the layers still work
    assert len(dk) == 10 and gk.sync_status() == 0


def test_serving_loop(kvc):
    """Prompt, decode steps that accumulate weights, an eviction whenever the budget
    is exceeded, more steps: against a float64 model of the same loop on the stored
    rows (the choice is checked on the GPU's own weights, the rest by allowance)."""
    from tree_cases import terms  # noqa: F401  (the reference reads the layers' own rows)
    import synth

    B, H, rep, D, S0, budget = 2, 2, 4, 128, 260, 200
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", B, H, D, S0, 7, dev=DEV, capacity=400)
    first = torch.tensor([0, 30], dtype=torch.int32, device=DEV)
    w = torch.zeros(B, H, 400, device=DEV)
    g = torch.Generator().manual_seed(1)
    new = synth.kv_spectral(B, H, 16, D, alpha=0.6, seed=99, tensor=0, dtype="f16")
    N, at = 32, 0
    for step in range(16):
        q = torch.randn(B, H * rep, N, D, generator=g)
        w0 = w.clone()
        o = kvc.attend_window(gk, gv, q.to(DEV), window=150, sinks=4, first=first, weights=w)
        S = len(gk)
        want, tol, ww, wtol = window_cases.reference(gk, rk, gv, rv, q.double().numpy(), D ** -0.5, 150, 4,
                                                     first.tolist(), w0.double().cpu().numpy())
        window_cases.check(o, want, tol, f"out of step {step}")
        window_cases.check(w[:, :, :S], ww, wtol, f"weights of step {step}")
        if S > budget:
            bk, bv, wh, f = _rows(gk), _rows(gv), w.cpu().numpy(), first.tolist()
            index, first = kvc.evict(gk, gv, w[:, :, :S], budget - 8, sinks=4, recent=32, first=first)
            want = np.stack([[evicted(wh[b, h, :S], budget - 8, 4, 32, f[b]) for h in range(H)]
                             for b in range(B)])
            _check(index, None, gk, bk, want)
            _check(index, None, gv, bv, want)
            assert bool((w[:, :, budget - 8:] == 0).all())
        gk.append(new[:, :, at:at + 1].to(DEV))
        gv.append(new[:, :, at:at + 1].to(DEV))
        at, N = at + 1, 1
