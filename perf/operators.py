"""Measured cases of the speculative-decoding operators of the quantised cache.

Three operators that work on stored rows (packed codes and their fp16 side
words) of key and value layers:

  attend_tree  attention of N drafted tokens per sequence over the cache, the
               drafted tokens being its last N rows, under a tree mask;
  gather       rows of one layer appended to another one: a prompt forked into
               beams, beams reordered, a cache compacted to chosen tokens;
  accept       the accepted ones among the last N (drafted) rows moved up, the
               others dropped.

``run`` computes each either in plain torch operations on the packed rows, or,
where ``own`` is true, through the package's public calls on layers that hold
the same rows.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the tiny test layer: four drafted tokens on a short prompt, all latency
        dict(name="tree tiny", op="attend_tree", B=1, H=2, rep=2, D=64, S=84, N=4, keys="uniform",
             kbits=0, values="int8", q="f32", out="f16", mask="tree", pad=False),
        # a padded batch with odd sizes everywhere, some drafted rows unused
        dict(name="tree ragged", op="attend_tree", B=3, H=5, rep=3, D=64, S=1777, N=7,
             keys="codebook", kbits=4, values="uniform", q="bf16", out="bf16", mask="holes", pad=True),
        # Llama-3-8B-like layer, fitted bases for keys and values, a tree of 16 drafts
        dict(name="tree llama", op="attend_tree", B=8, H=8, rep=4, D=128, S=4096, N=16,
             keys="uniform", kbits=0, values="uniform", q="bf16", out="bf16", mask="tree", pad=False),
        # one long sequence, five drafts in a chain: few rows, a long axis
        dict(name="tree long", op="attend_tree", B=1, H=8, rep=4, D=128, S=130001, N=5,
             keys="codebook", kbits=3, values="int8", q="f16", out="f16", mask="chain", pad=False),
        # TurboQuant-style serving batch, eight drafts
        dict(name="tree turboquant", op="attend_tree", B=16, H=8, rep=4, D=128, S=16384, N=8,
             keys="codebook", kbits=3, values="int8", q="f16", out="f16", mask="tree", pad=False),
        # the same batch with a wide tree: the most arithmetic
        dict(name="tree wide", op="attend_tree", B=16, H=8, rep=4, D=128, S=16384, N=32,
             keys="codebook", kbits=3, values="int8", q="bf16", out="bf16", mask="tree", pad=True),
        # a Llama-3-8B-like prompt of one sequence forked into eight beams
        dict(name="fork beams", op="gather", src_B=1, B=8, H=8, D=128, S=4096, n=4096, have=0,
             layer="uniform", kbits=0, rows="all"),
        # beams reordered: every value row of a serving batch moves
        dict(name="reorder values", op="gather", src_B=16, B=16, H=8, D=128, S=16384, n=16384,
             have=0, layer="int8", kbits=0, rows="all"),
        # a long key cache compacted to the third of its tokens that a policy keeps
        dict(name="compact keys", op="gather", src_B=16, B=16, H=8, D=128, S=16384, n=5461,
             have=77, layer="codebook", kbits=3, rows="chosen"),
        # three of eight drafts accepted on a short cache, all latency
        dict(name="accept small", op="accept", B=1, H=8, D=128, S=512, N=8, n=3, layer="int8",
             kbits=0),
        # verification of a wide tree in a serving batch
        dict(name="accept wide", op="accept", B=16, H=8, D=128, S=2048, N=64, n=17,
             layer="codebook", kbits=3),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend_tree", "attend_tree", "attend_tree", "gather", "gather", "accept"])
    D = rng.choice([64, 128, 128])
    H = rng.randint(1, 8)
    if op == "attend_tree":
        B, rep, N = _log(rng, 1, 16), rng.choice([1, 2, 3, 4, 5, 8]), _log(rng, 1, 40)
        # at most the arithmetic of the largest listed case
        top = 16 * 8 * 128 * 16384 // (B * H * rep * N)
        S = _log(rng, max(N, 1), max(N, min(131072, top, 16 * 8 * 16384 // (B * H))))
        keys = rng.choice(["codebook", "uniform"])
        return dict(op=op, B=B, H=H, rep=rep, D=D, S=S, N=N, keys=keys,
                    kbits=rng.choice([2, 3, 4]) if keys == "codebook" else 0,
                    values=rng.choice(["int8", "int8", "uniform"]), q=rng.choice(["f32", "f16", "bf16"]),
                    out=rng.choice(["f16", "bf16"]), mask=rng.choice(["tree", "chain", "holes"]),
                    pad=rng.random() < 0.3)
    layer = rng.choice(["codebook", "uniform", "int8"])
    kbits = rng.choice([2, 3, 4]) if layer == "codebook" else 0
    if op == "gather":
        B = _log(rng, 1, 16)
        src_B = rng.randint(1, B)
        S = _log(rng, 1, 16384)
        rows = rng.choice(["all", "chosen"])
        n = S if rows == "all" else rng.randint(1, S)
        return dict(op=op, src_B=src_B, B=B, H=H, D=D, S=S, n=n, have=rng.choice([0, 1, 77, 500]),
                    layer=layer, kbits=kbits, rows=rows)
    N = _log(rng, 1, 96)
    return dict(op=op, B=_log(rng, 1, 16), H=H, D=D, S=_log(rng, 1, 4096), N=N, n=rng.randint(1, N),
                layer=layer, kbits=kbits)


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
    """A layer of the package that holds these rows (S of them)."""
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


def _mask(kind, B, N, g, dev):
    """Which drafted token sees which: None for a chain, else bool [B, N, N]."""
    if kind == "chain":
        return None
    eye = torch.eye(N, dtype=torch.bool, device=dev)
    m = torch.zeros(B, N, N, dtype=torch.bool, device=dev)
    for i in range(N):  # a token's parent is an earlier one, or the last token of the context
        u = torch.rand(B, generator=g, device=dev)
        if i:
            parent = (u * (i + 1)).long() - 1
            m[:, i] = m[torch.arange(B, device=dev), parent.clamp(min=0)] & (parent >= 0)[:, None]
        m[:, i] |= eye[i]
    if kind == "holes":  # a quarter of the rows is not used
        m &= (torch.rand(B, N, 1, generator=g, device=dev) > 0.25)
    return m


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    c = dict(case)
    B, H, D = c["B"], c["H"], c["D"]
    if c["op"] == "attend_tree":
        S, N, Hq = c["S"], c["N"], c["H"] * c["rep"]
        st = dict(c, k=_rows(c["keys"], c["kbits"], B, H, S, D, g, dev),
                  v=_rows(c["values"], 0, B, H, S, D, g, dev))
        # queries as a projection leaves them: [B, N, heads, D], heads moved forward as a view
        q = torch.randn(B, N, Hq, D, generator=g, device=dev).to(DTYPES[c["q"]])
        st["queries"] = q.transpose(1, 2)
        st["tree"] = _mask(c["mask"], B, N, g, dev)
        st["first"] = None
        if c["pad"]:  # left padding: up to half of the context, the whole of it once
            ctx = S - N
            f = (torch.rand(B, generator=g, device=dev) * (ctx // 2 + 1)).int()
            f[B - 1] = ctx
            st["first"] = f
        if own:
            st["klayer"] = _layer(st["k"], B, H, D, S, S)
            st["vlayer"] = _layer(st["v"], B, H, D, S, S, c["out"])
        return st
    if c["op"] == "gather":
        rows = _rows(c["layer"], c["kbits"], c["src_B"], H, c["S"], D, g, dev)
        st = dict(c, src=rows)
        st["parent"] = None
        if not (c["src_B"] == B and c["rows"] == "chosen"):
            st["parent"] = torch.randint(0, c["src_B"], (B,), generator=g, device=dev, dtype=torch.int32)
        st["index"] = None
        if c["rows"] == "chosen":
            st["index"] = torch.stack([torch.randperm(c["S"], generator=g, device=dev)[:c["n"]].sort()[0]
                                       for _ in range(B)]).int()
        P = rows["packed"].shape[-1]
        have = torch.randint(0, 256, (B * H, c["have"], P), generator=g, device=dev, dtype=torch.uint8)
        hs = None if rows["side"] is None else torch.rand(B * H, c["have"], generator=g, device=dev).half()
        st["have_rows"] = dict(rows, packed=have, side=hs)
        if own:
            st["slayer"] = _layer(rows, c["src_B"], H, D, c["S"], c["S"])
            st["dlayer"] = _layer(st["have_rows"], B, H, D, c["have"] + c["n"], c["have"])
            st["rows_out"] = _views(st["dlayer"], c["have"] + c["n"])
        else:
            st["dst"] = torch.empty(B * H, c["have"] + c["n"], P, dtype=torch.uint8, device=dev)
            st["dst"][:, :c["have"]] = have
            if hs is not None:
                st["dst_side"] = torch.empty(B * H, c["have"] + c["n"], dtype=torch.float16, device=dev)
                st["dst_side"][:, :c["have"]] = hs
        return st
    rows = _rows(c["layer"], c["kbits"], B, H, c["S"] + c["N"], D, g, dev)
    base = dict(rows, packed=rows["packed"][:, :c["S"]].contiguous(),
                side=None if rows["side"] is None else rows["side"][:, :c["S"]].contiguous())
    drafts = dict(rows, packed=rows["packed"][:, c["S"]:].contiguous(),
                  side=None if rows["side"] is None else rows["side"][:, c["S"]:].contiguous())
    st = dict(c, base=base, drafts=drafts)
    st["index"] = torch.stack([torch.randperm(c["N"], generator=g, device=dev)[:c["n"]].sort()[0]
                               for _ in range(B)]).int()
    if own:
        st["layer_"] = _layer(base, B, H, D, c["S"] + c["N"], c["S"])
        st["dlayer"] = _layer(drafts, B, H, D, c["N"], c["N"])
        st["rows_out"] = _views(st["layer_"], c["S"] + c["n"])
    else:
        P = rows["packed"].shape[-1]
        st["dst"] = torch.empty(B * H, c["S"] + c["N"], P, dtype=torch.uint8, device=dev)
        st["dst"][:, :c["S"]] = base["packed"]
        if rows["side"] is not None:
            st["dst_side"] = torch.empty(B * H, c["S"] + c["N"], dtype=torch.float16, device=dev)
            st["dst_side"][:, :c["S"]] = base["side"]
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


def _decode(rows, B, H, D):
    """The rows that the codes stand for, [B, H, S, D] in fp32."""
    p = rows["packed"]
    ns, S, _ = p.shape
    if rows["kind"] == "int8":
        return (p.view(torch.int8).float() * rows["side"].float().unsqueeze(-1)).view(B, H, S, D)
    if rows["kind"] == "codebook":
        u = rows["levels"][_unpack(p, rows["kbits"], D).int()]
        return (torch.matmul(u, rows["V"].T) * rows["side"].float().unsqueeze(-1)).view(B, H, S, D)
    parts, at = [], 0
    for w in (8, 4, 2):
        m = rows["bits"].count(w)
        parts.append(_unpack(p[..., at:at + m * w // 8], w, m))
        at += m * w // 8
    z = torch.cat(parts, -1).view(B, H, S, rows["r"])
    z = rows["lo"][:, None] + z * rows["step"][:, None]
    return torch.matmul(z, rows["V"].transpose(-1, -2)) + rows["mean"][:, None]


def _attend_plain(st):
    B, H, rep, D, S, N = (st[k] for k in ("B", "H", "rep", "D", "S", "N"))
    K = _decode(st["k"], B, H, D)
    V = _decode(st["v"], B, H, D)
    dev, ctx = K.device, S - N
    seen = torch.ones(B, N, S, dtype=torch.bool, device=dev)
    if st["first"] is not None:
        seen[:, :, :ctx] = (torch.arange(ctx, device=dev) >= st["first"][:, None])[:, None]
    seen[:, :, ctx:] = st["tree"] if st["tree"] is not None else torch.tril(seen.new_ones(N, N))
    q = st["queries"].float().reshape(B, H, rep * N, D)
    s = torch.matmul(q, K.transpose(-1, -2)).view(B, H, rep, N, S) / math.sqrt(D)
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - top.masked_fill(top == -math.inf, 0.0))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, H, rep * N, S), V).view(B, H, rep, N, D) / total.clamp_min(1e-30)
    return o.reshape(B, H * rep, N, D).to(DTYPES[st["out"]])


def _gather_plain(st):
    B, H, S, n, have = st["B"], st["H"], st["S"], st["n"], st["have"]
    out = {}
    for part, key in (("dst", "packed"), ("dst_side", "side")):
        if st["src"][key] is None:
            continue
        x = st["src"][key]
        x = x.view(st["src_B"], H, S, *x.shape[2:])
        if st["parent"] is not None:
            x = x[st["parent"].long()]
        if st["index"] is not None:
            at = st["index"].long()
            x = x[torch.arange(B, device=x.device)[:, None, None],
                  torch.arange(H, device=x.device)[:, None], at[:, None]]
        st[part].view(B, H, have + n, *x.shape[3:])[:, :, have:] = x
        out[key] = st[part]
    return out


def _accept_plain(st):
    B, H, S, N, n = st["B"], st["H"], st["S"], st["N"], st["n"]
    out = {}
    for part, key in (("dst", "packed"), ("dst_side", "side")):
        if st["drafts"][key] is None:
            continue
        buf = st[part]
        buf[:, S:] = st["drafts"][key]
        x = buf.view(B, H, S + N, *buf.shape[2:])
        at = S + st["index"].long()
        x[:, :, S:S + n] = x[torch.arange(B, device=x.device)[:, None, None],
                             torch.arange(H, device=x.device)[:, None], at[:, None]]
        out[key] = buf[:, :S + n]
    return out


def run(st):
    if st["op"] == "attend_tree":
        if not own:
            return _attend_plain(st)
        import rank_quantized_kv_gb300 as kvc

        return kvc.attend_tree(st["klayer"], st["vlayer"], st["queries"], mask=st["tree"],
                               first=st["first"])
    if st["op"] == "gather":
        if not own:
            return _gather_plain(st)
        d = st["dlayer"]
        d.trim(len(d) - st["have"])
        d.gather(st["slayer"], parent=st["parent"], index=st["index"])
        p, s = st["rows_out"]
        return {"packed": p} if s is None else {"packed": p, "side": s}
    if not own:
        return _accept_plain(st)
    lay = st["layer_"]
    lay.trim(len(lay) - st["S"])
    lay.gather(st["dlayer"])          # the drafted rows join the cache
    lay.accept(st["index"], st["N"])  # and the accepted ones stay
    p, s = st["rows_out"]
    return {"packed": p} if s is None else {"packed": p, "side": s}


def _row_bytes(kind, kbits, D):
    """Packed bytes and side bytes of a stored row."""
    if kind == "int8":
        return D, 2
    if kind == "codebook":
        return D * kbits // 8, 2
    return sum(_widths(D)) // 8, 0


def work(case):
    c = case
    B, H, D = c["B"], c["H"], c["D"]
    if c["op"] == "attend_tree":
        S, N, rows = c["S"], c["N"], c["B"] * c["H"] * c["rep"] * c["N"]
        stored = B * H * S * (sum(_row_bytes(c["keys"], c["kbits"], D)) + sum(_row_bytes(c["values"], 0, D)))
        small = rows * D * (4 if c["q"] == "f32" else 2) + rows * D * 2
        small += B * N * N if c["mask"] != "chain" else 0
        # scores and weighted sums cost a product per stored component: the latent's, or the head's
        # D; a basis is applied to the queries and to the weighted mean latents alone
        r = len(_widths(D))
        kw, vw = (r if c["keys"] == "uniform" else D), (r if c["values"] == "uniform" else D)
        flops = 2 * rows * S * (kw + vw) + 2 * rows * D * kw
        flops += 2 * rows * D * vw if c["values"] == "uniform" else 0
        return dict(bytes=stored + small, flops=flops)
    row = sum(_row_bytes(c["layer"], c["kbits"], D))
    if c["op"] == "gather":
        # beams that share a parent share its rows: they are read once
        read = min(c["src_B"], B) * H * c["n"] * row
        idx = 4 * B * c["n"] if c["rows"] == "chosen" else 4 * B
        return dict(bytes=read + B * H * c["n"] * row + idx, flops=0)
    # the drafted rows written to the cache, the accepted ones read and written
    return dict(bytes=2 * B * H * (c["N"] + c["n"]) * row + 4 * B * c["n"], flops=0)


def exact(case, seed):
    """Attention in 64 bits, slot by slot, the codes read as bit fields of whole words."""
    if case["op"] != "attend_tree":
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
    ar = torch.arange(N, device=dev)
    for b in range(B):
        start = int(st["first"][b]) if st["first"] is not None else 0
        tree = st["tree"][b] if st["tree"] is not None else ar[:, None] >= ar
        hidden = torch.cat([(torch.arange(S - N, device=dev) < start).expand(N, -1), ~tree], 1)
        for h in range(H):
            K, V = rows64(st["k"], b * H + h), rows64(st["v"], b * H + h)
            for x in range(h * rep, (h + 1) * rep):
                s = st["queries"][b, x].double() @ K.T / D ** 0.5
                s[hidden] = -math.inf
                p = torch.exp(s - s.max(1, keepdim=True)[0])
                o = (p @ V) / p.sum(1, keepdim=True)
                out[b, x] = torch.where(hidden.all(1)[:, None], torch.zeros_like(o), o)
    return out
