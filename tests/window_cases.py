"""Shared by the tests of windowed attention and eviction: the float64 result on
the layers' own stored rows and the error that the kernels' roundings allow.

Output, per element, with p the float64 weights and every value row split into the
components the kernels sum (v_t = c + sum_j T_tj e_j), as for tree attention:
  half a step of the output type, relative to the output;
  (2^-11 + 2 delta) sum_t p_t sum_j |T_tj e_jd|: a weight may be rounded to fp16,
    and a score that is off by delta (in nats) moves a weight and the sum that
    divides it by a factor e^delta each;
  S 2^-31 max_t sum_j |T_tj e_jd|: weights below fp16's normal range;
  2^-18 of the absolute terms: fp32 sums of at most 2^17 terms in blocks.

delta = eps max_t scale sum_j a_j |T_tj| over the visible tokens, T and e now the
keys' components and a_j = sum_i |q_i e_ji|.  A score is a sum of at most 256 + 48
products in fp32 (256 components, 48 for the projection u = V^T q in shares), each
step off by 2^-24, and its operands are held to 22 bits at least: eps = 2^-15 covers
304 2^-24 + 2 2^-22.  Where no weights are asked for, codebook keys may carry their
centroids in fp16: eps = 2^-11 + 2^-15.

Weights, per token: sum over rows of p (2 delta + 2^-18 + rows 2^-24), the exponential
(2 units), the division and the sums; 2^-22 of decay times the old weight."""
import math

import numpy as np

from oracle.attend import attend_tree_rows, window_visible

from tree_cases import terms

OUT_EPS = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def reference(gk, rk, gv, rv, q, scale, window=0, sinks=0, first=None, weights=None, decay=1.0):
    """(out, allowance) [B, Hq, N, D] of q (float64), and the same for weights [B, H, S]."""
    B, Hq, N, D = q.shape
    H, S = gk.H, len(gk)
    rep = Hq // H
    eps = 2.0 ** -15
    if weights is None and getattr(rk, "mode", "codebook") != "uniform":
        eps += 2.0 ** -11
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    acc, wtol = np.zeros((B, H, S)), np.zeros((B, H, S))
    for b in range(B):
        vis = window_visible(N, S, window, sinks, 0 if first is None else int(first[b]))
        for h in range(H):
            K, TK, EK = terms(gk, rk, b * H + h)
            V, TV, EV = terms(gv, rv, b * H + h)
            av = np.abs(TV)
            for x in range(h * rep, (h + 1) * rep):
                o, p = attend_tree_rows(q[b, x], K, V, scale, vis)
                logit = scale * ((np.abs(q[b, x]) @ np.abs(EK).T) @ np.abs(TK).T)
                delta = eps * np.max(np.where(vis, logit, 0.0), axis=1, initial=0.0)
                terms_v = (p @ av) @ np.abs(EV)
                most = (av.max(0) if len(av) else np.zeros(av.shape[1])) @ np.abs(EV)
                tol[b, x] = (OUT_EPS[gv.out_dtype] * np.abs(o)
                             + (2.0 ** -11 + 2 * delta[:, None] + 2.0 ** -18) * terms_v
                             + S * 2.0 ** -31 * most + 2.0 ** -18 * (np.abs(o) + terms_v) + 2.0 ** -25)
                tol[b, x][~vis.any(1)] = 0.0  # a row that sees nothing is exactly zero
                out[b, x] = o
                acc[b, h] += p.sum(0)
                wtol[b, h] += (p * (2 * delta[:, None] + 2.0 ** -18 + rep * N * 2.0 ** -24)).sum(0)
    if weights is None:
        return out, tol, None, None
    old = decay * weights[:, :, :S] if decay else np.zeros_like(acc)
    return out, tol, old + acc, wtol + 2.0 ** -22 * np.abs(old) + 2.0 ** -120


def check(o, want, tol, what):
    err = np.abs(o.double().cpu().numpy() - want)
    assert np.all(err <= tol), (what, float(np.max(err / np.maximum(tol, 1e-300))))
