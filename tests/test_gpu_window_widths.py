"""Windowed attention and its weights over uniform keys of every number of packed
positions that the kernels tell apart (up to 32, 48, 64 and 128), widths from one to
eight bits in any order, another layout in every head; against the float64 oracle
within the allowance of window_cases.py."""
import math

import numpy as np
import pytest
import torch

import synth
import window_cases
from kvc_cases import oracle_kwargs
from oracle import codec, fit
from oracle.layer import OracleLayer

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
D = 128

# components by width: {width: count}; a width's components fill chunks of eight
WIDTHS = {8: {4: 5}, 16: {4: 16}, 32: {8: 8, 3: 13, 1: 3}, 40: {8: 4, 4: 20, 2: 8}, 48: {8: 7, 3: 17, 1: 16},
          56: {2: 56}, 120: {8: 120}, 64: {8: 3, 4: 40, 1: 9}, 80: {8: 3, 2: 65}, 128: {8: 1, 1: 120}}


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rank_quantized_kv_gb300 as kvc

    kvc.load_library()
    return kvc


@pytest.mark.parametrize("positions", sorted(WIDTHS))
@pytest.mark.parametrize("B,rep,N,S", [(1, 3, 1, 333), (1, 4, 2, 90), (1, 4, 40, 333), (10, 4, 8, 2100)])
def test_widths(kvc, positions, B, rep, N, S):
    counts = WIDTHS[positions]
    assert sum((n + 7) // 8 * 8 for n in counts.values()) == positions
    H, seed = 2, 31 * positions + S + N
    rng = np.random.default_rng(seed)
    xk = synth.kv_spectral(B, H, S, D, alpha=0.7, seed=seed, tensor=0, n_outliers=2, dtype="f16")
    xv = synth.kv_spectral(B, H, S, D, alpha=0.5, seed=seed + 1, tensor=1, dtype="f16")
    flat = np.concatenate([np.full(n, w) for w, n in counts.items()]).astype(np.uint8)
    r, V, mean, bits, lo, step = len(flat), [], [], [], [], []
    for s in range(B * H):
        x = xk.double().numpy()[s // H, s % H, :256]
        m, _, U = fit.pca_fit(x)
        v32, m32 = U[:, :r].astype(np.float32), m.astype(np.float32)
        b = rng.permutation(flat)
        a, st = fit.uniform_params(codec.project(x, m32, v32), b)
        V.append(v32), mean.append(m32), bits.append(b), lo.append(a.astype(np.float32)), step.append(st.astype(np.float32))
    p = dict(V=np.stack(V), mean=np.stack(mean), bits=np.stack(bits), qmin=np.stack(lo), qstep=np.stack(step),
             basis_of=np.arange(B * H))
    gk = kvc.KVCacheLayer("uniform", B, H, D, in_dtype="f16", capacity=S, device=DEV, **p)
    gv = kvc.KVCacheLayer("int8", B, H, D, in_dtype="f16", capacity=S, device=DEV)
    rk, rv = OracleLayer("uniform", B, H, D, **oracle_kwargs(p)), OracleLayer("int8", B, H, D)
    gk.append(xk.to(DEV))
    gv.append(xv.to(DEV))
    q = torch.randn(B, H * rep, N, D, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    w0 = torch.rand(B, H, S, generator=torch.Generator().manual_seed(seed))
    w = w0.to(DEV)
    o = kvc.attend_window(gk, gv, q.to(DEV), window=120, sinks=9, weights=w, decay=0.5)
    plain = kvc.attend_window(gk, gv, q.to(DEV), window=120, sinks=9)
    want, tol, ww, wtol = window_cases.reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(D), 120, 9, None,
                                                 w0.double().numpy(), 0.5)
    window_cases.check(o, want, tol, "out")
    window_cases.check(plain, want, tol, "out without weights")
    window_cases.check(w, ww, wtol, "weights")
    assert gk.sync_status() == 0
