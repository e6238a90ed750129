"""Tree attention over the whole range of key norms and query sizes: scores of
unit spread from norms of 1e-3 to fp16's largest, against the float64 oracle.

The allowance is that of tree_cases.py with the scores' error delta (in nats)
taken from what the kernels round, as the largest over the visible tokens of

  scale |sum_j u_j n (c'_j - c_j)|, u = V^T q: the centroids c' are the fp16
    values nearest to m c over m, m being the common scale that brings all
    levels closest to fp16 values (computed here as the library does);
  2^-19 scale max_j |u_j| sum_j |n c_j|: a row's key weights are multiplied by
    a power of two that brings the largest to 2^-6 .. 2^14, and what their two
    fp16 pieces leave is at most 2^-25;
  2^-18 scale sum_j |u_j n c_j|: 22 bits of a weight, fp32 products and sums;

and 2^-30 in place of 2^-31 for the smallest weights, as the value scales are
taken relative to a power of two of up to twice the largest."""
import math

import numpy as np
import pytest
import torch

import tree_cases
from kvc_cases import fit_codebook, oracle_kwargs
from oracle import codec
from oracle.attend import attend_tree_rows, tree_visible
from oracle.layer import OracleLayer
from tree_cases import check, make_layers, random_tree, terms

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


def rounded_centroids(c):
    """c as the tensor-core kernel holds it: fp16 values of m c, over m."""
    c = np.asarray(c, dtype=np.float32)
    _, e = np.frexp(np.abs(c).max())
    steps = 4096 * 8 // max(len(c), 8)
    f = np.float32(0.5) + np.float32(0.5) * np.arange(steps, dtype=np.float32) / np.float32(steps)
    m = (np.float32(2.0 ** (5 - int(e))) * f).astype(np.float32)
    v = m[:, None] * c[None]
    d = v.astype(np.float16).astype(np.float64) - v.astype(np.float64)
    m = m[np.argmin((d * d).sum(1) / m.astype(np.float64) ** 2)]
    return (m * c).astype(np.float16).astype(np.float64) / float(m)


def tight_reference(gk, rk, gv, rv, q, scale, N, first=None, mask=None):
    """As tree_cases.reference, for codebook keys, with the allowance above."""
    B, Hq, _, D = q.shape
    H, S = gk.H, len(gk)
    rep = Hq // H
    out_eps = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[gv.out_dtype]
    move = rounded_centroids(rk.codebook) - rk.codebook
    got = {}
    for b in range(B):
        vis = tree_visible(N, S, 0 if first is None else max(int(first[b]), 0),
                           None if mask is None else mask[b])
        for h in range(H):
            slot = b * H + h
            rows, side = gk.slot_rows(slot)
            rows = rows.cpu().numpy()
            n = side.cpu().numpy().view(np.float16)[:, 0].astype(np.float64)[:, None]
            codes = codec.unpack_rows(rows, rk.bits[0])
            K = rk.decode(slot, rows, n[:, 0].astype(np.float16))
            V, TV, EV = terms(gv, rv, slot)
            av = np.abs(TV)
            for x in range(h * rep, (h + 1) * rep):
                o, p = attend_tree_rows(q[b, x], K, V, scale, vis)
                u = q[b, x] @ rk.V[0]
                t = n * rk.codebook[codes]
                err = (np.abs(u @ (n * move[codes]).T)
                       + 2.0 ** -19 * np.abs(u).max(1)[:, None] * np.abs(t).sum(1)[None]
                       + 2.0 ** -18 * (np.abs(u) @ np.abs(t).T))
                delta = scale * np.max(np.where(vis, err, 0.0), axis=1, initial=0.0)
                terms_v = (p @ av) @ np.abs(EV)
                most = av.max(0) @ np.abs(EV)
                tol = (out_eps * np.abs(o) + (2.0 ** -11 + 2 * delta[:, None] + 2.0 ** -18) * terms_v
                       + S * 2.0 ** -30 * most + 2.0 ** -18 * (np.abs(o) + np.abs(terms_v)) + 2.0 ** -25)
                tol[~vis.any(1)] = 0.0
                got[b, x] = (o, tol)
    return got


def key_layers(kvc, B, H, D, S, bits, norm, seed):
    """Codebook keys of about the given norm under int8 values."""
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", B, H, D, 0, seed, bits=bits, capacity=S, dev=DEV)
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(B, H, S, D, generator=g)
    k = k / k.norm(dim=-1, keepdim=True) * norm * (0.5 + 0.5 * torch.rand(B, H, S, 1, generator=g))
    gk.append(k.half().to(DEV))
    gv.append(torch.randn(B, H, S, D, generator=g).half().to(DEV))
    return gk, gv, rk, rv


def unit_queries(B, Hq, N, D, norm, seed):
    """Queries that give such keys scores of a spread of about 1.5 (D^-1/2 scale)."""
    return torch.randn(B, Hq, N, D, generator=torch.Generator().manual_seed(seed)) * (2 * math.sqrt(D) / norm)


@pytest.mark.parametrize("norm", [1e-3, 1.0, 1e3, 1e4, 6e4])
@pytest.mark.parametrize("D,bits", [(128, 3), (64, 2), (128, 8)])
@pytest.mark.parametrize("rep,N", [(2, 4), (4, 8), (4, 15), (8, 16)])
def test_key_norms(kvc, norm, D, bits, rep, N):
    B, H, S = 1, 2, 500
    gk, gv, rk, rv = key_layers(kvc, B, H, D, S, bits, norm, 300 + D + bits)
    q = unit_queries(B, H * rep, N, D, norm, 17)
    mask = random_tree(np.random.default_rng(N), B, N)
    o = kvc.attend_tree(gk, gv, q.to(DEV), mask=torch.from_numpy(mask).to(DEV))
    check(o, tight_reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(D), N, mask=mask))


@pytest.mark.parametrize("norm", [10.0, 6e4])
@pytest.mark.parametrize("rep,N", [(2, 4), (4, 15), (8, 16)])
def test_rows_of_very_different_sizes(kvc, norm, rep, N):
    """Query rows of one head apart by up to 2^60, rows of zeros among them: each
    row is right, and rows of zeros change no other row."""
    B, H, D, S = 1, 1, 128, 700
    gk, gv, rk, rv = key_layers(kvc, B, H, D, S, 3, norm, 41)
    q = unit_queries(B, rep, N, D, norm, 18)
    q[0, 0, 1] *= 2.0 ** -30
    q[0, 1, 2] *= 2.0 ** -12
    q[0, 1, 0] *= 2.0 ** 4
    q[0, 1, 1] *= 2.0 ** -60
    o = kvc.attend_tree(gk, gv, q.to(DEV))
    check(o, tight_reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(D), N))
    q[0, 0, 1] = q[0, 1, 1] = q[0, 1, 2] = 0
    a = kvc.attend_tree(gk, gv, q.to(DEV))
    check(a, tight_reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(D), N))
    q[0, 0, 1] = q[0, 1, 1] = q[0, 1, 2] = q[0, 0, 0]
    b = kvc.attend_tree(gk, gv, q.to(DEV))
    keep = [(0, 0), (0, 2), (0, 3), (1, 0), (1, 3)]
    assert all(torch.equal(a[0, x, i], b[0, x, i]) for x, i in keep)


@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_uniform_keys_and_very_small_and_large_queries(kvc, size):
    """All query rows far from 1 with a scale that brings the scores back to it."""
    B, H, rep, D, S, N = 1, 2, 2, 64, 300, 5
    gk, gv, rk, rv = make_layers(kvc, "uniform", "uniform", B, H, D, S, 77, dev=DEV)
    q = torch.randn(B, H * rep, N, D, generator=torch.Generator().manual_seed(3)) * size
    scale = float(np.float32(1 / (size * math.sqrt(D))))
    o = kvc.attend_tree(gk, gv, q.to(DEV), scale=scale)
    check(o, tree_cases.reference(gk, rk, gv, rv, q.double().numpy(), scale, N))


@pytest.mark.parametrize("vmode", ["int8", "uniform"])
@pytest.mark.parametrize("D", [128, 64, 96])
def test_two_bit_codebooks(kvc, vmode, D):
    gk, gv, rk, rv = make_layers(kvc, "codebook", vmode, 2, 2, D, 400, 55, bits=2, dev=DEV)
    q = torch.randn(2, 6, 6, D, generator=torch.Generator().manual_seed(5))
    o = kvc.attend_tree(gk, gv, q.to(DEV))
    check(o, tight_reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(D), 6))


def test_rounded_centroids_are_near(kvc):
    """The table's own error: at most half an fp16 step of the level."""
    for bits in (1, 2, 3, 4):
        c = fit_codebook(128, bits)["codebook"].astype(np.float64)
        assert np.all(np.abs(rounded_centroids(c) - c) <= 2.0 ** -11 * np.abs(c) * (1 + 2.0 ** -20))


@pytest.mark.parametrize("size", [2.0 ** -124, 2.0 ** 100])
def test_very_small_and_large_codebooks(kvc, size):
    """Centroids at the ends of fp32's range under queries that bring the scores back."""
    B, H, rep, D, S, N = 1, 2, 2, 64, 300, 4
    p = fit_codebook(D, 3)
    p["codebook"] = (p["codebook"] * np.float32(size)).astype(np.float32)
    gk = kvc.KVCacheLayer("codebook", B, H, D, in_dtype="f16", capacity=S, device=DEV,
                          path=tree_cases.PATH[0], **p)
    rk = OracleLayer("codebook", B, H, D, **oracle_kwargs(p))
    _, gv, _, rv = make_layers(kvc, "codebook", "int8", B, H, D, S, 88, dev=DEV)
    g = torch.Generator().manual_seed(4)
    gk.append(torch.randn(B, H, S, D, generator=g).half().to(DEV))
    q = torch.randn(B, H * rep, N, D, generator=g) * (0.5 / size)
    o = kvc.attend_tree(gk, gv, q.to(DEV))
    check(o, tree_cases.reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(D), N))


@pytest.mark.parametrize("kmode,vmode", [("uniform", "uniform"), ("uniform", "int8"), ("codebook", "uniform"),
                                         ("codebook", "int8")])
@pytest.mark.parametrize("H,rep,N", [(4, 128, 50), (4, 35, 64)])
def test_jobs_of_different_sizes_in_turn(kvc, kmode, vmode, H, rep, N):
    """Many short jobs, several to a CTA, with query heads of ordinary, very large and
    very small size, alone and together in a job: none takes another's factors."""
    B, D, S = 1, 64, 130
    gk, gv, rk, rv = make_layers(kvc, kmode, vmode, B, H, D, S, 90, dev=DEV)
    g = torch.Generator().manual_seed(6)
    size = 2.0 ** torch.tensor([0, 0, 18, -24])[torch.randint(0, 4, (H * rep // 4 + 1,), generator=g)]
    q = torch.randn(B, H * rep, N, D, generator=g) * size.repeat_interleave(4)[:H * rep, None, None]
    o = kvc.attend_tree(gk, gv, q.to(DEV))
    check(o, tree_cases.reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(D), N))
