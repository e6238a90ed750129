"""Rows moved between and inside layers (gather, accept): byte for byte against
plain indexing, and a speculative step put together from them."""
import math

import numpy as np
import pytest
import torch

import synth
from kvc_cases import fit_codebook, fit_group, fit_uniform
from tree_cases import check, make_layers, random_tree, reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rank_quantized_kv_gb300 as kvc

    kvc.load_library()
    return kvc


# kind -> (D, parameters for one batch entry of H heads); row bytes 1 to 128, side words 0 to 8
def _params(kind, H):
    rng = np.random.default_rng(1)
    if kind == "int8":
        return "int8", 128, {}
    if kind == "int8 odd":
        return "int8", 37, {}
    if kind == "codebook":
        return "codebook", 128, fit_codebook(128)
    if kind == "codebook odd":
        return "codebook", 24, fit_codebook(24, 1)
    if kind == "group":
        x = rng.standard_normal((1, H, 200, 32))
        p = fit_group(x, 2, 48)
        return "group", 32, p
    if kind == "prod":
        return "codebook", 64, dict(fit_codebook(64, 2), sketch=rng.standard_normal((32, 64)),
                                    outlier_channels=np.tile(np.array([[1, 8, 50]], dtype=np.int32), (H, 1)),
                                    split_from=3)
    bits = {"uniform": [8] * 4 + [4] * 20 + [2] * 8, "uniform odd": [8, 4, 4, 3, 1, 1], "uniform wide": [8] * 24,
            "uniform none": [0, 0]}[kind]
    r = len(bits)
    return "uniform", 32, dict(V=rng.standard_normal((H, 32, r)), mean=rng.standard_normal((H, 32)),
                               bits=np.tile(np.array(bits, dtype=np.uint8), (H, 1)), qmin=-np.ones((H, r)),
                               qstep=np.full((H, r), 0.1), basis_of=np.arange(H))


KINDS = ["int8", "int8 odd", "codebook", "codebook odd", "group", "prod", "uniform", "uniform odd",
         "uniform wide", "uniform none"]


def _layer(kvc, kind, B, H, cap, T, seed, **kw):
    mode, D, p = _params(kind, H)
    p = dict(p, **kw)
    if "basis_of" in p:
        p["basis_of"] = np.tile(p["basis_of"], B)
    if "outlier_channels" in p:
        p["outlier_channels"] = np.tile(p["outlier_channels"], (B, 1))
    lay = kvc.KVCacheLayer(mode, B, H, D, in_dtype="f16", capacity=cap, device=DEV, **p)
    g = torch.Generator(device=DEV).manual_seed(seed)
    lay.store.copy_(torch.randint(0, 256, lay.store.shape, generator=g, device=DEV, dtype=torch.uint8))
    if T:
        lay.append(torch.randn(B, H, T, D, generator=g, device=DEV).half())
    return lay


def _regions(lay, cap=None):
    """Every slot's payload and side bytes up to the capacity, as numpy rows."""
    cap = cap or lay.capacity
    store = lay.store.cpu().numpy()
    got = []
    for s in range(lay.n_slots):
        a = lay.slot_layout(s)
        for o, w in ((a["payload_offset"], a["row_bytes"]), (a["side_offset"], a["side_bytes"])):
            got.append(store[o:o + cap * w].reshape(cap, w).copy())
    return got


def _gather_ref(dst, src, have, n, parent, index, start, B, Bs, per):
    """What dst's regions become; per: regions of a batch entry."""
    want = [r.copy() for r in dst]
    for b in range(B):
        sb = b if parent is None else int(parent[b])
        rows = np.arange(start, start + n) if index is None else index[b]
        for i in range(per):
            if 0 <= sb < Bs:
                for j, s in enumerate(rows):
                    if s >= 0 and (index is None or s < len(src[0])):
                        want[b * per + i][have + j] = src[sb * per + i][s]
    return want


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Bs,B,S,have,n,how", [
    (2, 2, 300, 0, 300, "all"), (1, 3, 65, 7, 65, "parent"), (3, 2, 200, 3, 50, "start"),
    (2, 2, 129, 5, 40, "index"), (2, 5, 400, 1, 333, "both"), (1, 1, 1, 0, 1, "all"), (1, 4, 3, 2, 1, "both"),
])
def test_gather_moves_bytes(kvc, kind, Bs, B, S, have, n, how):
    H = 2
    src = _layer(kvc, kind, Bs, H, S + 3, S, 1)
    dst = _layer(kvc, kind, B, H, have + n + 9, have, 2)
    rng = np.random.default_rng(S)
    parent = rng.integers(0, Bs, B).astype(np.int32) if how in ("parent", "both", "start") else None
    index = rng.integers(0, S, (B, n)).astype(np.int32) if how in ("index", "both") else None
    start = 11 if how == "start" else 0
    before, rows = _regions(dst), [r[:S] for r in _regions(src)]
    dst.gather(src, parent=None if parent is None else torch.from_numpy(parent).to(DEV),
               index=None if index is None else torch.from_numpy(index).to(DEV), start=start,
               n=None if index is not None else n)
    assert len(dst) == have + n and dst.sync_status() == 0
    want = _gather_ref(before, rows, have, n, parent, index, start, B, Bs, len(before) // B)
    for a, w in zip(_regions(dst), want):
        assert np.array_equal(a, w)  # rows around the range are left as they were


def test_gather_bad_entries_move_nothing(kvc):
    """Entries outside the source: their rows keep their bytes, the others move,
    and sync_status reports it once."""
    src = _layer(kvc, "codebook", 2, 2, 40, 33, 3)
    dst = _layer(kvc, "codebook", 3, 2, 30, 4, 4)
    parent = np.array([1, 2, 0], dtype=np.int32)
    index = np.random.default_rng(0).integers(0, 33, (3, 20)).astype(np.int32)
    index[0, 3], index[2, 7], index[2, 19] = -1, 33, 2 ** 31 - 1
    before, rows = _regions(dst), [r[:33] for r in _regions(src)]
    dst.gather(src, parent=torch.from_numpy(parent).to(DEV), index=torch.from_numpy(index).to(DEV))
    assert dst.sync_status() == -6 and dst.sync_status() == 0
    for a, w in zip(_regions(dst), _gather_ref(before, rows, 4, 20, parent, index, 0, 3, 2, len(before) // 3)):
        assert np.array_equal(a, w)


def test_gather_refusals(kvc):
    src = _layer(kvc, "uniform", 2, 2, 20, 10, 5)
    dst = _layer(kvc, "uniform", 2, 2, 12, 4, 6)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)

    def refused(status, d, s, **kw):
        n = len(d)
        with pytest.raises(kvc.KvcError) as e:
            d.gather(s, **kw)
        assert e.value.status == status and len(d) == n

    refused(-1, src, src)                                              # the same layer
    refused(-3, dst, src, n=9)                                         # capacity
    refused(-1, dst, src, start=5, n=6)                                # past the source's end
    refused(-1, dst, src, start=-1, n=2)
    refused(-1, dst, src, n=-1)
    refused(-1, dst, src, start=1, index=torch.zeros(2, 2, dtype=torch.int32, device=DEV))
    refused(-1, _layer(kvc, "uniform", 3, 2, 20, 0, 7), src)           # other batch without parent
    refused(-1, dst, _layer(kvc, "uniform odd", 2, 2, 20, 10, 8), n=1)  # other parameters
    refused(-1, dst, _layer(kvc, "uniform", 2, 2, 20, 10, 8, mean=np.zeros((2, 32))), n=1)
    refused(-1, dst, _layer(kvc, "uniform", 2, 2, 20, 10, 8, basis_of=np.array([1, 0])), n=1)  # other bases
    refused(-1, dst, src, n=2, parent=zero.cpu())
    per_entry = dict(V=np.random.default_rng(1).standard_normal((4, 32, 8)), mean=None,
                     bits=np.full((4, 8), 4, dtype=np.uint8), qmin=np.zeros((4, 8)), qstep=np.ones((4, 8)))
    a, b = (kvc.KVCacheLayer("uniform", 2, 2, 32, in_dtype="f16", capacity=8, device=DEV,
                             basis_of=np.arange(4), **per_entry) for _ in range(2))
    a.append(torch.randn(2, 2, 3, 32, device=DEV).half())
    refused(-1, b, a, parent=zero)                                     # a basis per batch entry: rows may not change it
    b.gather(a)                                                        # but may keep it
    assert len(b) == 3
    for bad in (dict(parent=zero.long()), dict(parent=zero[:1]), dict(index=zero),
                dict(index=torch.zeros(2, 3, dtype=torch.int32, device=DEV), n=2)):
        with pytest.raises(ValueError):
            dst.gather(src, **bad)
    n = len(dst)
    dst.gather(src, n=0)
    assert len(dst) == n


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,S,N,n,order", [(2, 50, 8, 3, "up"), (1, 5, 5, 5, "any"), (3, 200, 130, 77, "up"),
                                           (2, 64, 33, 33, "any"), (1, 9, 1, 1, "up"), (2, 30, 16, 9, "repeat"),
                                           (1, 4000, 3900, 3000, "up")])
def test_accept_moves_bytes(kvc, kind, B, S, N, n, order):
    lay = _layer(kvc, kind, B, 2, S + 4, S, 9)
    rng = np.random.default_rng(N)
    idx = np.stack([rng.permutation(N)[:n] if order != "repeat" else rng.integers(0, N, n) for _ in range(B)])
    idx = (np.sort(idx, 1) if order == "up" else idx).astype(np.int32)
    before = _regions(lay)
    lay.accept(torch.from_numpy(idx).to(DEV), N)
    assert len(lay) == S - N + n and lay.sync_status() == 0
    per = len(before) // B
    for i, (a, w) in enumerate(zip(_regions(lay), before)):
        w = w.copy()
        w[S - N:S - N + n] = w[S - N + idx[i // per]]
        assert np.array_equal(a, w)


def test_accept_edges_and_refusals(kvc):
    lay = _layer(kvc, "codebook", 2, 2, 40, 30, 10)
    idx = torch.tensor([[0, 5], [9, -1]], dtype=torch.int32, device=DEV)
    before = _regions(lay)
    lay.accept(idx, 8)  # 9 and -1 lie outside the 8: their rows stay
    assert len(lay) == 24 and lay.sync_status() == -6 and lay.sync_status() == 0
    per = len(before) // 2
    for i, (a, w) in enumerate(zip(_regions(lay), before)):
        w = w.copy()
        if i < per:
            w[23] = before[i][27]
        assert np.array_equal(a, w)
    for args in ((idx, 25), (idx, 1), (idx, -1), (idx.cpu(), 8)):
        with pytest.raises(kvc.KvcError) as e:
            lay.accept(*args)
        assert e.value.status == -1 and len(lay) == 24
    for bad in (idx.long(), idx[:1], idx[:, 0], idx.t()):
        with pytest.raises(ValueError):
            lay.accept(bad, 8)
    lay.accept(torch.empty(2, 0, dtype=torch.int32, device=DEV), 4)  # none accepted: a trim
    assert len(lay) == 20


def test_large_offsets(kvc):
    """Rows past 2^32 bytes into the store."""
    B, H, cap = 1, 40, 1 << 20
    src = kvc.KVCacheLayer("int8", B, H, 128, in_dtype="f16", capacity=cap, device=DEV)
    src.append(torch.randn(B, 1, 1, 128, device=DEV).half().expand(B, H, cap, 128))
    a = src.slot_layout(H - 1)
    assert a["payload_offset"] > 2 ** 32
    src.store[a["payload_offset"]:a["payload_offset"] + cap * 128] = torch.randint(0, 256, (cap * 128,), device=DEV,
                                                                                   dtype=torch.uint8)
    dst = kvc.KVCacheLayer("int8", B, H, 128, in_dtype="f16", capacity=cap, device=DEV)
    dst.gather(src, start=5)
    assert len(dst) == cap - 5
    got, want = dst.slot_rows(H - 1), src.slot_rows(H - 1)
    assert torch.equal(got[0], want[0][5:]) and torch.equal(got[1], want[1][5:])
    idx = torch.tensor([[1, 3, 9]], dtype=torch.int32, device=DEV)
    keep = got[0][-10:].clone()
    dst.accept(idx, 10)
    assert torch.equal(dst.slot_rows(H - 1)[0][-3:], keep[[1, 3, 9]])


def test_captured_and_replayed(kvc):
    """gather and accept in a graph: a replay moves what the layers hold then."""
    src = _layer(kvc, "int8", 1, 2, 64, 50, 11)
    dst = _layer(kvc, "int8", 2, 2, 64, 0, 12)
    parent = torch.zeros(2, dtype=torch.int32, device=DEV)
    idx = torch.tensor([[2, 3, 4], [0, 6, 7]], dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dst.gather(src, parent=parent)
        dst.accept(idx, 8)
    src.store.random_(0, 256)
    g.replay()
    torch.cuda.synchronize()
    assert len(dst) == 45
    for s in range(4):
        want = src.slot_rows(s % 2)[0][42:][idx[s // 2].long()]
        assert torch.equal(dst.slot_rows(s)[0][42:], want)
        assert torch.equal(dst.slot_rows(s)[0][:42], src.slot_rows(s % 2)[0][:42])


@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "uniform"), ("prod", "int8")])
def test_speculative_step(kvc, kmode, vmode):
    """A prompt forked into two beams, a tree of drafts appended and scored, the
    accepted path kept, the next step on top: everything equals layers that held
    the accepted tokens from the start."""
    H, D, S, N, n, rep = 2, 64, 150, 7, 3, 2
    one = {}
    if kmode == "uniform":  # a basis per head, shared by the batch
        x = synth.kv_spectral(1, H, 300, D, alpha=0.7, seed=5, tensor=0, dtype="f16")
        one["k"] = fit_uniform(x.double().numpy(), 256, 32, [0, 2, 4, 8], 96)
        one["v"] = fit_uniform(x.double().numpy() * 0.5, 256, 32, [0, 2, 4, 8], 128)
    elif kmode == "prod":
        one["k"] = dict(fit_codebook(D, 2), sketch=np.random.default_rng(1).standard_normal((32, D)),
                        outlier_channels=np.tile(np.array([[3, 17]], dtype=np.int32), (H, 1)), split_from=4)
        one["v"] = {}
    else:
        one["k"], one["v"] = fit_codebook(D), {}

    def layer(which, mode, B, cap=200):
        p = dict(one[which])
        for key in ("basis_of", "outlier_channels"):
            if key in p:
                p[key] = np.concatenate([p[key]] * B)
        return kvc.KVCacheLayer("codebook" if mode == "prod" else mode, B, H, D, in_dtype="f16", capacity=cap,
                                device=DEV, **p)

    g = torch.Generator(device=DEV).manual_seed(3)
    rnd = lambda B, T: torch.randn(B, H, T, D, generator=g, device=DEV).half()  # noqa: E731
    prompt, drafts, nxt = (rnd(1, S), rnd(1, S)), (rnd(2, N), rnd(2, N)), (rnd(2, 1), rnd(2, 1))
    mask = random_tree(np.random.default_rng(4), 2, N)
    path = torch.tensor([[0, 2, 5], [1, 3, 6]], dtype=torch.int32, device=DEV)
    q = torch.randn(2, H * rep, N, D, generator=g, device=DEV)
    lay, ref = [], []
    for i, (which, mode) in enumerate((("k", kmode), ("v", vmode))):
        base = layer(which, mode, 1)
        base.append(prompt[i])
        two = layer(which, mode, 2)
        two.gather(base, parent=torch.zeros(2, dtype=torch.int32, device=DEV))
        two.append(drafts[i])
        lay.append(two)
        want = layer(which, mode, 2)
        want.append(prompt[i].expand(2, H, S, D).contiguous())
        kept = drafts[i][torch.arange(2, device=DEV)[:, None], :, path.long()].transpose(1, 2).contiguous()
        want.append(kept)
        ref.append(want)
    out = kvc.attend_tree(*lay, q, mask=torch.from_numpy(mask).to(DEV))
    # draft by draft: the drafts a row sees, appended alone, then a decode step
    for b, i in ((0, 0), (0, 5), (1, 6)):
        alone = []
        for which, mode, x, y in (("k", kmode, prompt[0], drafts[0]), ("v", vmode, prompt[1], drafts[1])):
            one_l = layer(which, mode, 2)
            one_l.append(x.expand(2, H, S, D).contiguous())
            one_l.append(y[:, :, torch.from_numpy(np.flatnonzero(mask[b, i])).to(DEV)].contiguous())
            alone.append(one_l)
        single = kvc.attend_tree(*alone, q[:, :, i:i + 1])
        assert torch.allclose(out[b, :, i].float(), single[b, :, 0].float(), rtol=2e-3, atol=2e-3)
    for a, w in zip(lay, ref):
        a.accept(path, N)
        assert len(a) == len(w) == S + n and a.sync_status() == 0
        for s in range(a.n_slots):
            for x, y in zip(a.slot_rows(s), w.slot_rows(s)):
                assert x is None and y is None or torch.equal(x, y)
    for i in range(2):
        lay[i].append(nxt[i])
        ref[i].append(nxt[i])
    q1 = torch.randn(2, H * rep, 1, D, generator=g, device=DEV)
    assert torch.equal(kvc.attend_tree(*lay, q1), kvc.attend_tree(*ref, q1))
