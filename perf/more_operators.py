"""Measured cases of the operators that keep a quantised cache within a budget.

Three uses of two public calls on key and value layers (packed codes and fp16
side words):

  window   attention of the last N stored tokens over a sliding window and the
           first tokens (sinks), which stay visible;
  weights  the same attention, and for every stored token the softmax weight
           that it received, added to an accumulator per key/value head;
  evict    the tokens of least accumulated weight dropped from both layers,
           the sinks and the most recent tokens kept in any case.

``run`` computes each either in plain torch operations on the packed rows, or,
where ``own`` is true, through the package's public calls on layers that hold
the same rows.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _attention(name, B, H, rep, D, S, N, window, sinks, keys, kbits, values, q, out, pad=False,
               decay=-1.0):
    """A case of attention; decay below 0: no weights, 0: weights set, 1: added."""
    return dict(name=name, op="window" if decay < 0 else "weights", B=B, H=H, rep=rep, D=D, S=S,
                N=N, window=window, sinks=sinks, keys=keys, kbits=kbits, values=values, q=q,
                out=out, pad=pad, decay=decay)


def _evict(name, B, H, D, S, keep, sinks, recent, keys, kbits, values, pad=False, place="into"):
    return dict(name=name, op="evict", B=B, H=H, D=D, S=S, keep=keep, sinks=sinks, recent=recent,
                keys=keys, kbits=kbits, values=values, pad=pad, place=place)


def listed():
    return [
        # the tiny test layer, one token on a short prompt: all latency
        _attention("window tiny", 1, 2, 2, 64, 84, 1, 32, 4, "uniform", 0, "int8", "f32", "f16"),
        # a padded batch with odd sizes everywhere, seven tokens at once
        _attention("window ragged", 3, 5, 3, 64, 1777, 7, 500, 3, "codebook", 4, "uniform", "bf16",
                   "bf16", pad=True),
        # a decode step of a TurboQuant-style serving batch, a quarter of the context in the window
        _attention("window serving", 16, 8, 4, 128, 16384, 1, 4096, 4, "codebook", 3, "int8", "f16",
                   "f16"),
        # one long sequence, a wide window, fitted bases for keys and values: few rows, a long axis
        _attention("window long", 1, 8, 4, 128, 130001, 1, 100000, 64, "uniform", 0, "uniform",
                   "bf16", "bf16"),
        # a chunk of a long prompt appended to the cache: the most arithmetic
        _attention("window prompt", 1, 8, 4, 128, 8192, 2048, 2048, 4, "codebook", 3, "int8", "bf16",
                   "bf16"),
        # a decode step that keeps count of the weights, a short odd cache
        _attention("weights small", 2, 4, 4, 128, 513, 1, 0, 0, "codebook", 2, "int8", "f16", "f16",
                   decay=1.0),
        # the same of a serving batch over the whole context
        _attention("weights serving", 16, 8, 4, 128, 16384, 1, 0, 0, "codebook", 3, "int8", "f16",
                   "f16", decay=1.0),
        # the last 32 tokens of a Llama-3-8B-like prompt observe which of its tokens matter
        _attention("weights observe", 8, 8, 4, 128, 4096, 32, 0, 0, "uniform", 0, "uniform", "bf16",
                   "bf16", decay=0.0),
        # a short cache brought back to its budget in place
        _evict("evict small", 1, 8, 128, 600, 512, 4, 64, "codebook", 3, "int8", place="same"),
        # a padded batch with odd sizes, into smaller layers
        _evict("evict ragged", 3, 5, 64, 1777, 701, 3, 33, "uniform", 0, "uniform", pad=True),
        # the prompts of a serving batch cut to a quarter
        _evict("evict serving", 16, 8, 128, 16384, 4096, 4, 256, "codebook", 3, "int8"),
        # one long sequence cut to a quarter: few rows to share the selection among
        _evict("evict long", 1, 8, 128, 130001, 32768, 64, 1024, "uniform", 0, "int8"),
    ]


def _log(rng, lo, hi):
    hi = max(lo, hi)
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _nameless(case):
    del case["name"]
    return case


def draw(rng):
    op = rng.choice(["window", "window", "window", "weights", "weights", "evict", "evict"])
    D = rng.choice([64, 128, 128])
    B, H = _log(rng, 1, 16), rng.randint(1, 8)
    keys = rng.choice(["codebook", "uniform"])
    kbits = rng.choice([2, 3, 4]) if keys == "codebook" else 0
    values = rng.choice(["int8", "int8", "uniform"])
    pad = rng.random() < 0.3
    if op == "evict":
        S = _log(rng, 1, min(131072, 16 * 8 * 16384 // (B * H)))
        keep = rng.randint(1, S)
        sinks = min(keep, rng.choice([0, 1, 4, 64]))
        recent = rng.randint(0, keep - sinks)
        return _nameless(_evict("", B, H, D, S, keep, sinks, recent, keys, kbits, values, pad,
                                rng.choice(["into", "into", "same"])))
    rep = rng.choice([1, 2, 3, 4, 5, 8])
    # at most the scores of the largest listed case, and as many stored rows
    most = 8 * 4 * 2048 * 2048
    N = _log(rng, 1, rng.choice([1, 8, 64, 2048]))
    N = max(1, min(N, most // (B * H * rep * 64)))
    S = _log(rng, N, min(131072, 16 * 8 * 16384 // (B * H), most // (B * H * rep * N)))
    window = rng.choice([0, _log(rng, 1, S), _log(rng, 1, S)])
    decay = -1.0 if op == "window" else rng.choice([0.0, 1.0, 0.9])
    return _nameless(_attention("", B, H, rep, D, S, N, window, rng.choice([0, 1, 4, 64]), keys,
                                kbits, values, rng.choice(["f32", "f16", "bf16"]),
                                rng.choice(["f16", "bf16"]), pad, decay))


# ------------------------------------------------------------------ inputs

def _widths(D):
    """Widths of a uniform layer's components, as a fit with a budget of D bits leaves them."""
    u = D // 32
    return [8] * u + [4] * (5 * u) + [2] * (2 * u)


def _pack(codes, width):
    """Codes [..., k] of one width as bytes, least significant bit first."""
    if width == 8:
        return codes.to(torch.uint8)
    k = codes.shape[-1]
    shift = torch.arange(width, device=codes.device, dtype=torch.uint8)
    bits = ((codes.to(torch.uint8).unsqueeze(-1) >> shift) & 1).reshape(*codes.shape[:-1], k * width)
    place = 2 ** torch.arange(8, device=codes.device, dtype=torch.uint8)
    return (bits.view(*codes.shape[:-1], k * width // 8, 8) * place).sum(-1, dtype=torch.uint8)


def _rows(kind, kbits, B, H, S, D, g, dev):
    """Stored rows of a layer: packed [B*H, S, P] uint8 and side [B*H, S] fp16 (or None), with the
    frozen parameters they decode by; the codes are those of Gaussian rows."""
    ns = B * H
    if kind == "int8":
        v = torch.randn(ns, S, D, generator=g, device=dev)
        v += 0.5 * torch.randn(ns, 1, D, generator=g, device=dev)
        s = v.abs().amax(-1) / 127.0
        packed = (v / s.unsqueeze(-1)).round_().to(torch.int8).view(torch.uint8)
        return dict(kind=kind, packed=packed, side=s.half())
    if kind == "codebook":
        n_lev = 1 << kbits
        R = torch.linalg.qr(torch.randn(D, D, generator=g, device=dev, dtype=torch.float64))[0].float()
        # levels at the conditional means of equal parts of a Gaussian
        edge = torch.special.ndtri(torch.arange(1, n_lev, device=dev, dtype=torch.float64) / n_lev)
        dens = torch.cat([edge.new_zeros(1), torch.exp(-edge * edge / 2) / math.sqrt(2 * math.pi),
                          edge.new_zeros(1)])
        levels = (n_lev * (dens[:-1] - dens[1:]) / math.sqrt(D)).float()
        mids = (levels[1:] + levels[:-1]) / 2
        packed = torch.empty(ns, S, D * kbits // 8, dtype=torch.uint8, device=dev)
        norms = torch.empty(ns, S, dtype=torch.float16, device=dev)
        for a in range(0, ns, 16):
            z = torch.randn(min(16, ns - a), S, D, generator=g, device=dev)
            nrm = z.norm(dim=-1)
            packed[a:a + 16] = _pack(torch.bucketize(z / nrm.unsqueeze(-1), mids), kbits)
            norms[a:a + 16] = nrm.half()
        return dict(kind=kind, packed=packed, side=norms, V=R, levels=levels, kbits=kbits)
    bits = _widths(D)
    r = len(bits)
    V = torch.linalg.qr(torch.randn(H, D, r, generator=g, device=dev, dtype=torch.float64))[0].float()
    mean = 0.5 * torch.randn(H, D, generator=g, device=dev)
    sig = 4.0 / torch.arange(1, r + 1, device=dev, dtype=torch.float32).sqrt()
    qmax = torch.tensor([(1 << b) - 1 for b in bits], device=dev, dtype=torch.float32)
    step = (6 * sig / qmax).expand(H, r) * (0.9 + 0.2 * torch.rand(H, r, generator=g, device=dev))
    lo = -step * qmax / 2
    parts, k = [], 0
    for w in (8, 4, 2):
        m = bits.count(w)
        z = torch.randn(B, H, S, m, generator=g, device=dev) * sig[k:k + m]
        c = torch.round((z - lo[:, None, k:k + m]) / step[:, None, k:k + m])
        parts.append(_pack(torch.minimum(c.clamp_(min=0), qmax[k:k + m]).view(ns, S, m), w))
        k += m
    return dict(kind=kind, packed=torch.cat(parts, -1), side=None, V=V, mean=mean, bits=bits, lo=lo,
                step=step, r=r)


def _layer(rows, B, H, D, capacity, S, out="f16"):
    """A layer of the package that holds the first S of these rows."""
    import rank_quantized_kv_gb300 as kvc

    host = {}
    if rows["kind"] == "codebook":
        host = dict(V=rows["V"].cpu().numpy(), codebook=rows["levels"].cpu().numpy())
    elif rows["kind"] == "uniform":
        host = dict(V=rows["V"].cpu().numpy(), mean=rows["mean"].cpu().numpy(),
                    bits=np.tile(np.array(rows["bits"], dtype=np.uint8), (H, 1)),
                    qmin=rows["lo"].cpu().numpy(), qstep=rows["step"].cpu().numpy(),
                    basis_of=np.tile(np.arange(H), B))
    lay = kvc.KVCacheLayer(rows["kind"], B, H, D, in_dtype="f16", out_dtype=out, capacity=capacity,
                           device=rows["packed"].device, **host)
    if S:
        lay.append(torch.zeros(B, H, S, D, dtype=torch.float16, device=lay.device))
        p, s = _views(lay, S)
        p.copy_(rows["packed"])
        if s is not None:
            s.copy_(rows["side"])
    return lay


def _views(lay, n):
    """A layer's first n rows as views of its store: packed [slots, n, P], side [slots, n]."""
    ns = lay.n_slots
    a = lay.slot_layout(0)
    stride = (lay.slot_layout(1)["payload_offset"] - a["payload_offset"]) if ns > 1 else lay.store.numel()
    p = lay.store.as_strided((ns, n, a["row_bytes"]), (stride, a["row_bytes"], 1), a["payload_offset"])
    if not a["side_bytes"]:
        return p, None
    h = lay.store.view(torch.float16)
    return p, h.as_strided((ns, n), (stride // 2, a["side_bytes"] // 2), a["side_offset"] // 2)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    c = dict(case)
    B, H, D, S = c["B"], c["H"], c["D"], c["S"]
    st = dict(c, k=_rows(c["keys"], c["kbits"], B, H, S, D, g, dev),
              v=_rows(c["values"], 0, B, H, S, D, g, dev))
    st["first"] = None
    if c["pad"]:  # left padding: up to half of the tokens, all but the last one once
        f = (torch.rand(B, generator=g, device=dev) * (S // 2 + 1)).int()
        f[B - 1] = S - 1
        st["first"] = f
    if c["op"] != "evict":
        N, Hq = c["N"], H * c["rep"]
        # queries as a projection leaves them: [B, N, heads, D], heads moved forward as a view
        q = 1.5 * torch.randn(B, N, Hq, D, generator=g, device=dev)
        st["queries"] = q.to(DTYPES[c["q"]]).transpose(1, 2)
        if c["decay"] >= 0:  # what earlier steps added up, room for later tokens behind it
            st["w"] = torch.exp(torch.randn(B, H, S + 16, generator=g, device=dev)) / S
        if own:
            st["klayer"] = _layer(st["k"], B, H, D, S, S)
            st["vlayer"] = _layer(st["v"], B, H, D, S, S, c["out"])
        return st
    # accumulated weights: a long tail of light tokens, some that no query has seen yet
    w = torch.exp(2 * torch.randn(B, H, S, generator=g, device=dev))
    st["w"] = w * (torch.rand(B, H, S, generator=g, device=dev) > 0.1)
    n = c["keep"]
    if own:
        st["klayer"] = _layer(st["k"], B, H, D, S, S)
        st["vlayer"] = _layer(st["v"], B, H, D, S, S)
        room = n if c["place"] == "into" else S
        st["kdst"] = _layer(st["k"], B, H, D, room, 0)
        st["vdst"] = _layer(st["v"], B, H, D, room, 0)
        st["wdst"] = torch.zeros(B, H, room, device=dev)
        st["kdst"].gather(st["klayer"], n=n)  # so that the views below have rows to show
        st["vdst"].gather(st["vlayer"], n=n)
        st["rows_out"] = _views(st["kdst"], n) + _views(st["vdst"], n)
    return st


# ------------------------------------------------------------------ the plain forms

def _unpack(packed, width, k):
    """k codes of one width from bytes [..., ceil(k width / 8)]."""
    if width == 8:
        return packed.float()
    dev = packed.device
    bits = (packed.unsqueeze(-1) >> torch.arange(8, device=dev, dtype=torch.uint8)) & 1
    bits = bits.view(*packed.shape[:-1], packed.shape[-1] * 8)[..., :k * width]
    place = 2 ** torch.arange(width, device=dev, dtype=torch.uint8)
    return (bits.view(*packed.shape[:-1], k, width) * place).sum(-1, dtype=torch.uint8).float()


def _decode(rows, at, B, H, D):
    """The rows numbered `at` that the codes stand for, [B, H, len(at), D] in fp32."""
    p = rows["packed"][:, at]
    side = None if rows["side"] is None else rows["side"][:, at].float().unsqueeze(-1)
    ns, S, _ = p.shape
    if rows["kind"] == "int8":
        return (p.view(torch.int8).float() * side).view(B, H, S, D)
    if rows["kind"] == "codebook":
        u = rows["levels"][_unpack(p, rows["kbits"], D).int()]
        return (torch.matmul(u, rows["V"].T) * side).view(B, H, S, D)
    parts, byte = [], 0
    for w in (8, 4, 2):
        m = rows["bits"].count(w)
        parts.append(_unpack(p[..., byte:byte + m * w // 8], w, m))
        byte += m * w // 8
    z = torch.cat(parts, -1).view(B, H, S, rows["r"])
    z = rows["lo"][:, None] + z * rows["step"][:, None]
    return torch.matmul(z, rows["V"].transpose(-1, -2)) + rows["mean"][:, None]


def _attend_plain(st):
    B, H, rep, D, S, N, window, sinks = (st[k] for k in ("B", "H", "rep", "D", "S", "N", "window", "sinks"))
    dev = st["queries"].device
    at = torch.arange(S, device=dev)
    if window and st["first"] is None:  # the tokens that some query sees, and no others
        at = at[(at < sinks) | (at > S - N - window)]
    K, V = _decode(st["k"], at, B, H, D), _decode(st["v"], at, B, H, D)
    pos = torch.arange(S - N, S, device=dev)[:, None]
    first = st["first"] if st["first"] is not None else torch.zeros(B, dtype=torch.int32, device=dev)
    first = first[:, None, None]
    seen = (at <= pos) & (at >= first)
    if window:
        seen = seen & ((at > pos - window) | (at < first + sinks))
    q = st["queries"].float().reshape(B, H, rep * N, D)
    s = torch.matmul(q, K.transpose(-1, -2)).view(B, H, rep, N, len(at)) / math.sqrt(D)
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - top.masked_fill(top == -math.inf, 0.0))
    total = e.sum(-1, keepdim=True).clamp_min(1e-30)
    o = torch.matmul(e.view(B, H, rep * N, len(at)), V).view(B, H, rep, N, D) / total
    o = o.reshape(B, H * rep, N, D).to(DTYPES[st["out"]])
    if st["decay"] < 0:
        return o
    w = st["w"].clone()
    w[:, :, :S] *= st["decay"]
    w[:, :, at] += (e / total).sum((2, 3))
    return {"out": o, "weights": w}


def _evict_plain(st):
    B, H, S, n, w = st["B"], st["H"], st["S"], st["keep"], st["w"]
    at = torch.arange(S, device=w.device)
    first = st["first"] if st["first"] is not None else torch.zeros(B, dtype=torch.int32, device=w.device)
    f = first[:, None, None]
    rank = w.masked_fill((at >= f) & ((at < f + st["sinks"]) | (at >= S - st["recent"])), math.inf)
    rank = rank.masked_fill((at < f).expand_as(w), -math.inf)
    index = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :n].sort(-1)[0]
    out = {"index": index.int(), "first": (n - (S - first)).clamp_min(0).int(),
           "weights": torch.gather(w, 2, index)}
    for part, rows in (("k", st["k"]), ("v", st["v"])):
        flat = index.view(B * H, n, 1)
        out[part + "packed"] = torch.gather(rows["packed"], 1, flat.expand(-1, -1, rows["packed"].shape[-1]))
        if rows["side"] is not None:
            out[part + "side"] = torch.gather(rows["side"], 1, flat[..., 0])
    return out


def run(st):
    if not own:
        return _evict_plain(st) if st["op"] == "evict" else _attend_plain(st)
    import rank_quantized_kv_gb300 as kvc

    if st["op"] == "window":
        return kvc.attend_window(st["klayer"], st["vlayer"], st["queries"], window=st["window"],
                                 sinks=st["sinks"], first=st["first"])
    if st["op"] == "weights":
        w = st["w"].clone()
        o = kvc.attend_window(st["klayer"], st["vlayer"], st["queries"], window=st["window"],
                              sinks=st["sinks"], first=st["first"], weights=w, decay=st["decay"])
        return {"out": o, "weights": w}
    k, v, w, n = st["kdst"], st["vdst"], st["wdst"], st["keep"]
    k.trim(len(k))
    v.trim(len(v))
    if st["place"] == "into":
        index, first = kvc.evict(st["klayer"], st["vlayer"], st["w"], n, sinks=st["sinks"],
                                 recent=st["recent"], first=st["first"], into=(k, v, w))
    else:  # the layers that are evicted in place are filled again in every pass
        k.gather(st["klayer"])
        v.gather(st["vlayer"])
        w.copy_(st["w"])
        index, first = kvc.evict(k, v, w, n, sinks=st["sinks"], recent=st["recent"],
                                 first=st["first"])
    kp, ks, vp, vs = st["rows_out"]
    if first is None:  # nothing is padded, and nothing will be
        first = torch.zeros(st["B"], dtype=torch.int32, device=w.device)
    out = {"index": index, "first": first, "weights": w[:, :, :n], "kpacked": kp, "vpacked": vp}
    if ks is not None:
        out["kside"] = ks
    if vs is not None:
        out["vside"] = vs
    return out


def _row_bytes(kind, kbits, D):
    """Bytes of a stored row, packed codes and side words."""
    return D + 2 if kind == "int8" else D * kbits // 8 + 2 if kind == "codebook" else sum(_widths(D)) // 8


def _pairs(S, N, window, sinks):
    """Tokens that some query sees, and (query, token) pairs, without padding."""
    span = [min(p + 1, window) if window else p + 1 for p in range(S - N, S)]
    extra = [min(sinks, p + 1 - s) for p, s in zip(range(S - N, S), span)]
    low = min(p + 1 - s for p, s in zip(range(S - N, S), span))
    return S - low + min(sinks, low), sum(span) + sum(extra)


def work(case):
    c = case
    B, H, D, S = c["B"], c["H"], c["D"], c["S"]
    row = _row_bytes(c["keys"], c["kbits"], D) + _row_bytes(c["values"], 0, D)
    if c["op"] == "evict":
        # all weights read, the kept rows read and written with their weights and numbers
        return dict(bytes=B * H * (4 * S + c["keep"] * (2 * row + 8)), flops=0)
    N, rows = c["N"], B * H * c["rep"] * c["N"]
    tokens, pairs = _pairs(S, N, c["window"], c["sinks"])
    r = len(_widths(D))
    kw, vw = (r if c["keys"] == "uniform" else D), (r if c["values"] == "uniform" else D)
    nbytes = B * H * tokens * row + rows * D * (4 if c["q"] == "f32" else 2) + rows * D * 2
    if c["decay"] >= 0:  # set: written; added: read and written
        nbytes += B * H * tokens * (4 if c["decay"] == 0 else 8)
    # a product per stored component for scores and weighted sums; a basis is applied to the
    # queries and to the weighted mean latents alone
    flops = 2 * B * H * c["rep"] * pairs * (kw + vw) + 2 * rows * D * kw
    flops += 2 * rows * D * vw if c["values"] == "uniform" else 0
    return dict(bytes=nbytes, flops=flops)


def exact(case, seed):
    """Attention in 64 bits, slot by slot, the codes read as bit fields of whole words."""
    if case["op"] == "evict":
        return None  # whole rows move: there is nothing to round
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    B, H, rep, D, S, N = (st[k] for k in ("B", "H", "rep", "D", "S", "N"))
    dev = st["queries"].device

    def fields(p, first_bit, width, k):
        """k fields of `width` bits from bit `first_bit` of byte rows p [S, P], as integers."""
        p = torch.cat([p.long(), p.new_zeros(p.shape[0], 1).long()], 1)
        at = first_bit + width * torch.arange(k, device=dev)
        two = p[:, at // 8] + 256 * p[:, at // 8 + 1]
        return torch.div(two, 2 ** (at % 8), rounding_mode="floor") % 2 ** width

    def rows64(r, slot):
        p = r["packed"][slot]
        if r["kind"] == "int8":
            x = p.double()
            return torch.where(x > 127, x - 256, x) * r["side"][slot].double()[:, None]
        if r["kind"] == "codebook":
            u = r["levels"].double()[fields(p, 0, r["kbits"], D)]
            return r["side"][slot].double()[:, None] * (u @ r["V"].double().T)
        h, z, bit = slot % H, [], 0
        for k, w in enumerate(r["bits"]):
            z.append(fields(p, bit, w, 1)[:, 0].double() * r["step"][h, k].double() + r["lo"][h, k].double())
            bit += w
        return torch.stack(z, 1) @ r["V"][h].double().T + r["mean"][h].double()

    out = torch.zeros(B, H * rep, N, D, dtype=torch.float64, device=dev)
    acc = torch.zeros(B, H, S, dtype=torch.float64, device=dev)
    t = torch.arange(S, device=dev)
    for b in range(B):
        start = int(st["first"][b]) if st["first"] is not None else 0
        for h in range(H):
            K, V = rows64(st["k"], b * H + h), rows64(st["v"], b * H + h)
            for n0 in range(0, N, 256):
                pos = torch.arange(S - N + n0, min(S, S - N + n0 + 256), device=dev)[:, None]
                hidden = (t > pos) | (t < start)
                if st["window"]:
                    hidden |= (pos - t >= st["window"]) & (t - start >= st["sinks"])
                for x in range(h * rep, (h + 1) * rep):
                    s = st["queries"][b, x, n0:n0 + 256].double() @ K.T / D ** 0.5
                    s[hidden] = -math.inf
                    p = torch.softmax(s, 1)
                    p[hidden.all(1)] = 0.0
                    out[b, x, n0:n0 + 256] = p @ V
                    acc[b, h] += p.sum(0)
    if st["decay"] < 0:
        return out
    w = st["w"].double()
    w[:, :, :S] = w[:, :, :S] * st["decay"] + acc
    return {"out": out, "weights": w}
