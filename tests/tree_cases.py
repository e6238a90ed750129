"""Shared by the tests of tree attention: layers, the float64 result of their
own stored rows and the error that the kernels' roundings allow.

The allowance, per output element, with p the float64 weights and every value
row split into the components the kernels sum (v_t = c + sum_j T_tj e_j):

  half a step of the output type, relative to the output;
  (2^-11 + 2 delta) sum_t p_t sum_j |T_tj e_jd|: a weight is rounded to fp16
    (half a step: 2^-11), and a score that is off by delta (in nats) moves a
    weight and the sum that divides it by a factor e^delta each;
  S 2^-31 max_t sum_j |T_tj e_jd|: weights below fp16's normal range are off by
    at most 2^-25 where the sum of the weights is at least 2^6;
  2^-18 of the absolute terms: fp32 sums of at most 2^17 terms in blocks.

delta = eps max_t scale sum_j |q . e_j| |T_tj| over the visible tokens, with
eps = 2^-11 for codebook keys (their centroids are rounded to fp16) and 2^-18
for uniform keys (codes are exact in fp16, the key weights carry two fp16
pieces, sums are in fp32)."""
import math

import numpy as np
import torch

import synth
from oracle import codec, prod
from oracle.attend import attend_tree_rows, tree_visible
from oracle.layer import OracleLayer

from kvc_cases import fit_codebook, fit_uniform, oracle_kwargs

PATH = ["auto"]  # the kernels that the layers of make_layers use: a fixture sets it

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def make_layers(kvc, kmode, vmode, B, H, D, S, seed, out="f16", bits=3, capacity=None, dev=None):
    """Key and value layers of S appended tokens, with the oracle's twins."""
    cap = capacity or S
    xk = synth.kv_spectral(B, H, max(S, 2), D, alpha=0.7, seed=seed, tensor=0, n_outliers=2, dtype="f16")
    xv = synth.kv_spectral(B, H, max(S, 2), D, alpha=0.5, seed=seed + 1, tensor=1, dtype="f16")
    kx = {}
    if kmode == "uniform":
        pk = fit_uniform(xk.double().numpy(), min(max(S, 2), 256), min(32, D), [0, 1, 2, 3, 4, 8], D + D // 4)
    else:
        pk = fit_codebook(D, 2 if kmode == "prod" else min(bits, 4))
        if bits == 8 and kmode != "prod":  # 256 levels: evenly spaced will do
            pk["codebook"] = (np.linspace(-4, 4, 256) / math.sqrt(D)).astype(np.float32)
    if kmode == "prod":
        rng = np.random.default_rng(seed)
        kx = dict(sketch=rng.standard_normal((48, D)).astype(np.float32), split_from=5,
                  outlier_channels=np.stack([np.sort(rng.choice(D, 3, replace=False))
                                             for _ in range(B * H)]).astype(np.int32))
    pv = {} if vmode == "int8" else fit_uniform(xv.double().numpy(), min(max(S, 2), 256), min(40, D),
                                                [0, 1, 2, 3, 4, 8], 2 * D)
    gk = kvc.KVCacheLayer("codebook" if kmode == "prod" else kmode, B, H, D, in_dtype="f16",
                          capacity=cap, device=dev, path=PATH[0], **pk, **kx)
    gv = kvc.KVCacheLayer(vmode, B, H, D, in_dtype="f16", out_dtype=out, capacity=cap, device=dev, **pv)
    if kmode == "prod":
        rk = prod.ProdKeyLayer(B, H, D, R=pk["V"], centroids=pk["codebook"], S=kx["sketch"],
                               channels=kx["outlier_channels"], split_from=5)
    else:
        rk = OracleLayer(kmode, B, H, D, **oracle_kwargs(pk))
    rv = OracleLayer(vmode, B, H, D, **oracle_kwargs(pv))
    if S:
        gk.append(xk[:, :, :S].to(dev))
        gv.append(xv[:, :, :S].to(dev))
    return gk, gv, rk, rv


def terms(gl, rl, slot):
    """(decoded rows X [S, D], T [S, m], E [m, D]) with X = const + T E."""
    rows, side = gl.slot_rows(slot)
    rows = rows.cpu().numpy()
    D = gl.D
    sd = None if side is None else side.cpu().numpy().view(np.float16)
    if isinstance(rl, prod.ProdKeyLayer):
        e = rl.unpack(slot, rows, sd.reshape(rows.shape[0], -1))
        X = rl.decode(slot, e)
        T = [e["norm16"].astype(np.float64)[:, None] * rl.centroids[e["idx"]]]
        E = [rl.R.T]
        if rl.m:
            T.append(math.sqrt(math.pi / 2) / rl.m * e["gamma16"].astype(np.float64)[:, None]
                     * np.ones((1, rl.m)))
            E.append(rl.S)
        if rl.n_out:
            T.append(e["oscale16"].astype(np.float64)[:, None] * e["o8"].astype(np.float64))
            E.append(np.eye(D)[rl.channels[slot]])
        return X, np.concatenate(T, 1), np.concatenate(E, 0)
    if rl.mode == "int8":
        X = rl.decode(slot, rows, sd[:, 0])
        return X, X, np.eye(D)
    if rl.mode == "codebook":
        X = rl.decode(slot, rows, sd[:, 0])
        codes = codec.unpack_rows(rows, rl.bits[0])
        return X, sd[:, :1].astype(np.float64) * rl.codebook[codes], rl.V[0].T
    bsel = rl.basis_of[slot]
    bits = rl.bits[bsel]
    codes = codec.unpack_rows(rows, bits)
    keep = bits > 0
    half = 2.0 ** (np.maximum(bits, 1) - 1)
    T = ((codes - half) * rl.qstep[bsel])[:, keep]
    return rl.decode(slot, rows, None), T, rl.V[bsel].T[keep]


def reference(gk, rk, gv, rv, q, scale, N, first=None, mask=None, pairs=None):
    """{(b, hq): (out [N, D], allowance [N, D])} of q [B, Hq, N, D] (float64)."""
    B, Hq, _, D = q.shape
    H, S = gk.H, len(gk)
    rep = Hq // H
    eps = 2.0 ** -18 if getattr(rk, "mode", "") == "uniform" else 2.0 ** -11
    out_eps = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[gv.out_dtype]
    got = {}
    for b in range(B):
        vis = tree_visible(N, S, 0 if first is None else max(int(first[b]), 0),
                           None if mask is None else mask[b])
        for h in range(H):
            todo = [x for x in range(h * rep, (h + 1) * rep) if pairs is None or (b, x) in pairs]
            if not todo:
                continue
            K, TK, EK = terms(gk, rk, b * H + h)
            V, TV, EV = terms(gv, rv, b * H + h)
            av = np.abs(TV)
            for x in todo:
                o, p = attend_tree_rows(q[b, x], K, V, scale, vis)
                logit = scale * (np.abs(q[b, x] @ EK.T) @ np.abs(TK).T)
                delta = eps * np.max(np.where(vis, logit, 0.0), axis=1, initial=0.0)
                terms_v = (p @ av) @ np.abs(EV)
                most = (av.max(0) if len(av) else np.zeros(av.shape[1])) @ np.abs(EV)
                tol = (out_eps * np.abs(o) + (2.0 ** -11 + 2 * delta[:, None] + 2.0 ** -18) * terms_v
                       + S * 2.0 ** -31 * most + 2.0 ** -18 * (np.abs(o) + np.abs(terms_v)) + 2.0 ** -25)
                tol[~vis.any(1)] = 0.0  # a row that sees nothing is exactly zero
                got[b, x] = (o, tol)
    return got


def check(out, ref):
    o = out.float().cpu().numpy().astype(np.float64)
    for (b, x), (want, tol) in ref.items():
        err = np.abs(o[b, x] - want)
        assert np.all(err <= tol), (b, x, float(np.max(err / np.maximum(tol, 1e-300))))


def random_tree(rng, B, N, unused=0.0):
    """bool [B, N, N]: every draft sees itself and its ancestors; a share of the rows sees nothing."""
    m = np.zeros((B, N, N), dtype=bool)
    for b in range(B):
        for i in range(N):
            par = int(rng.integers(-1, i)) if i else -1
            if par >= 0:
                m[b, i] = m[b, par]
            m[b, i, i] = True
        m[b, rng.random(N) < unused] = False
    return m
