"""GPU parity of tree attention (kvc_attend_tree) against the float64 oracle on
the GPU's own stored rows, within the allowance derived in tree_cases.py."""
import concurrent.futures
import math
import threading

import numpy as np
import pytest
import torch

import tree_cases
from tree_cases import TORCH, check, make_layers, random_tree, reference

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
    """Every test on the tensor cores (where the layers allow it) and on the CUDA cores."""
    tree_cases.PATH[0] = request.param
    yield
    tree_cases.PATH[0] = "auto"


def _q(B, Hq, N, D, seed, dt="f32", scale=1.0):
    q = scale * torch.randn(B, Hq, N, D, generator=torch.Generator().manual_seed(seed))
    return q.to(TORCH[dt])


def _dev(a, dt=None):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _run(kvc, kmode, vmode, B, H, rep, D, S, N, dt="f32", out="f16", mask=None, first=None, bits=3,
         qscale=1.0, seed=None, pairs=None, **kw):
    seed = seed if seed is not None else 1000 + S + 7 * N + D
    gk, gv, rk, rv = make_layers(kvc, kmode, vmode, B, H, D, S, seed, out=out, bits=bits, dev=DEV)
    q = _q(B, H * rep, N, D, seed, dt, qscale)
    o = kvc.attend_tree(gk, gv, q.to(DEV), mask=_dev(mask), first=_dev(first), **kw)
    torch.cuda.synchronize()
    ref = reference(gk, rk, gv, rv, q.double().numpy(), kw.get("scale") or 1 / math.sqrt(D), N,
                    first, mask, pairs)
    check(o, ref)
    return gk, gv, q, o


@pytest.mark.parametrize("kmode,vmode,bits", [("codebook", "int8", 3), ("uniform", "uniform", 0),
                                              ("uniform", "int8", 0), ("codebook", "uniform", 4),
                                              ("codebook", "int8", 8), ("codebook", "int8", 1),
                                              ("prod", "int8", 2), ("prod", "uniform", 2)])
@pytest.mark.parametrize("D,rep,N,S", [(128, 4, 8, 700), (64, 2, 5, 131), (128, 1, 1, 257)])
def test_modes(kvc, kmode, vmode, bits, D, rep, N, S):
    rng = np.random.default_rng(N)
    _run(kvc, kmode, vmode, 2, 2, rep, D, S, N, bits=bits, mask=random_tree(rng, 2, N))


@pytest.mark.parametrize("D", [20, 32, 96, 200, 256])
@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "uniform")])
def test_head_sizes(kvc, kmode, vmode, D):
    if kmode == "codebook" and D % 4:
        pytest.skip("3-bit rows of whole bytes are not needed here")
    _run(kvc, kmode, vmode, 1, 2, 3, D, 300, 6)


@pytest.mark.parametrize("rep,N", [(1, 2), (3, 5), (5, 7), (8, 4), (8, 16), (4, 32), (2, 33), (4, 40), (16, 9),
                                   (1, 130), (7, 40)])
@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "uniform")])
def test_row_counts(kvc, kmode, vmode, rep, N):
    """Rows below, at and above one tile of rows, over several tiles of tokens."""
    rng = np.random.default_rng(rep * 100 + N)
    _run(kvc, kmode, vmode, 1, 2, rep, 128, 420, N, dt="bf16", mask=random_tree(rng, 1, N, unused=0.2))


@pytest.mark.parametrize("S,N", [(1, 1), (2, 2), (5, 5), (127, 3), (128, 3), (128, 128), (129, 3), (130, 3),
                                 (255, 1), (256, 40), (257, 130), (1025, 9)])
@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "uniform")])
def test_lengths(kvc, kmode, vmode, S, N):
    """Lengths at and around the tiles of 128 tokens, drafts across a tile's
    end, no context at all."""
    _run(kvc, kmode, vmode, 2, 1, 2, 64, S, N, dt="f16")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f16", "bf16"])
def test_types(kvc, dt, out):
    _run(kvc, "codebook", "int8", 1, 2, 2, 128, 300, 4, dt=dt, out=out)
    _run(kvc, "uniform", "uniform", 1, 2, 2, 128, 300, 4, dt=dt, out=out)


@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "uniform")])
def test_padded_batch(kvc, kmode, vmode):
    """Left padding from none to the whole context and beyond, rows that see
    nothing (zeros, whatever out held before), a padding that starts inside a tile."""
    B, H, rep, D, S, N = 6, 1, 4, 128, 700, 6
    first = np.array([0, -3, 150, 256, S - N, 10 ** 6], dtype=np.int32)
    rng = np.random.default_rng(3)
    mask = random_tree(rng, B, N, unused=0.4)
    mask[4, 2] = False
    mask[5] = False
    gk, gv, q, o = _run(kvc, kmode, vmode, B, H, rep, D, S, N, mask=mask, first=first)
    assert bool((o[5] == 0).all()) and bool((o[4, :, 2] == 0).all())
    out = torch.full_like(o, float("nan"))
    kvc.attend_tree(gk, gv, q.to(DEV), mask=_dev(mask), first=_dev(first), out=out)
    assert torch.equal(out, o)


@pytest.mark.parametrize("scale", [0.02, 3.0])
@pytest.mark.parametrize("kmode,vmode", [("codebook", "int8"), ("uniform", "int8"), ("uniform", "uniform")])
def test_scales(kvc, kmode, vmode, scale):
    """Flat and sharply peaked weights (the running maximum moves far)."""
    _run(kvc, kmode, vmode, 1, 2, 2, 128, 1500, 5, scale=scale)
    _run(kvc, kmode, vmode, 1, 2, 2, 128, 1500, 5, qscale=1e-5)


def test_rising_scores(kvc):
    """Keys whose scores rise along the sequence, so that every tile has a new maximum."""
    B, H, D, S, N = 1, 2, 64, 1200, 4
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", B, H, D, 0, 5, capacity=S, dev=DEV)
    g = torch.Generator().manual_seed(11)
    base = torch.randn(D, generator=g)
    ramp = torch.linspace(-4, 12, S)[None, None, :, None]
    k = (ramp * base + 0.3 * torch.randn(B, H, S, D, generator=g)).half()
    v = (torch.randn(B, H, S, D, generator=g) * torch.logspace(-2, 2, S)[None, None, :, None]).half()
    gk.append(k.to(DEV))
    gv.append(v.to(DEV))
    q = (base + 0.1 * torch.randn(B, 2 * H, N, D, generator=g)).float()
    o = kvc.attend_tree(gk, gv, q.to(DEV))
    check(o, reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(D), N))


def test_falling_values(kvc):
    """Value rows that shrink along the sequence, by 2^20 in all, under weights that grow."""
    B, H, D, S, N = 1, 2, 64, 900, 3
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", B, H, D, 0, 6, capacity=S, dev=DEV)
    g = torch.Generator().manual_seed(12)
    base = torch.randn(D, generator=g)
    k = torch.linspace(-2, 6, S)[None, None, :, None] * base + 0.3 * torch.randn(B, H, S, D, generator=g)
    v = torch.randn(B, H, S, D, generator=g) * torch.logspace(10, -10, S, base=2.0)[None, None, :, None]
    gk.append(k.half().to(DEV))
    gv.append(v.half().to(DEV))
    q = (base + 0.1 * torch.randn(B, 2 * H, N, D, generator=g)).float()
    o = kvc.attend_tree(gk, gv, q.to(DEV))
    check(o, reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(D), N))


@pytest.mark.parametrize("shared", [True, False])
def test_many_drafts(kvc, shared):
    """More drafts than the threads of a block, several words of mask bits a
    draft, jobs that begin inside a word."""
    B, H, rep, D, S, N = 2, 1, 2, 64, 700, 333
    mask = random_tree(np.random.default_rng(9), 1 if shared else B, N, unused=0.1)
    gk, gv, rk, rv = make_layers(kvc, "uniform", "int8", B, H, D, S, 91, dev=DEV)
    q = _q(B, H * rep, N, D, 9)
    o = kvc.attend_tree(gk, gv, q.to(DEV), mask=_dev(mask[0] if shared else mask))
    check(o, reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(D), N,
                       mask=np.repeat(mask, B, 0) if shared else mask))


def test_two_streams_at_once(kvc):
    """Calls that overlap on two streams, each with scratch of its own: the bits of calls one by one."""
    gk, gv, _, _ = make_layers(kvc, "codebook", "int8", 2, 2, 128, 4000, 95, dev=DEV)
    qs = [_q(2, 8, 5, 128, 100 + i).to(DEV) for i in range(2)]
    want = [kvc.attend_tree(gk, gv, q) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            got[i].append(kvc.attend_tree(gk, gv, qs[i], stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])


def test_dropped_components(kvc):
    """Bases of which no component is kept: rows of no bytes, equal scores, the mean row."""
    B, H, D, S, N = 1, 2, 64, 300, 3
    rng = np.random.default_rng(0)
    p = dict(V=rng.standard_normal((H, D, 4)), mean=rng.standard_normal((H, D)).astype(np.float32),
             bits=np.zeros((H, 4), dtype=np.uint8), qmin=np.zeros((H, 4)), qstep=np.ones((H, 4)),
             basis_of=np.arange(H))
    lay = [kvc.KVCacheLayer("uniform", B, H, D, in_dtype="f16", capacity=S, device=DEV,
                            path=tree_cases.PATH[0], **p) for _ in range(2)]
    for x in lay:
        x.append(torch.randn(B, H, S, D, device=DEV).half())
    o = kvc.attend_tree(*lay, _q(B, 2 * H, N, D, 3).to(DEV)).float().cpu().numpy()
    want = np.repeat(p["mean"], 2, 0)[None, :, None]
    assert np.all(np.abs(o - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -18 * np.abs(want) + 2.0 ** -25)


def test_one_draft_is_a_decode_step(kvc):
    """N = 1 without a mask gives what kvc.attend gives, up to the output's rounding."""
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", 2, 2, 128, 900, 21, dev=DEV)
    q = _q(2, 8, 1, 128, 4)
    a = kvc.attend(gk, gv, q[:, :, 0].contiguous().to(DEV)).float()
    b = kvc.attend_tree(gk, gv, q.to(DEV))
    ref = reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(128), 1)
    check(b, ref)
    assert float((a - b[:, :, 0].float()).abs().max()) <= 4e-3 * float(a.abs().max())


def test_what_hidden_tokens_hold_has_no_effect(kvc):
    """Infinities and NaN in the norms and scales of hidden tokens (padding, drafts
    behind the mask, rows behind the last token), and the largest codes."""
    B, H, D, S, N = 2, 2, 128, 400, 5
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", B, H, D, S, 31, capacity=S + 40, dev=DEV)
    q = _q(B, 2 * H, N, D, 5).to(DEV)
    first = torch.tensor([40, 133], dtype=torch.int32, device=DEV)
    mask = torch.eye(N, dtype=torch.bool).expand(B, N, N).contiguous()
    mask[:, :, 2] = False  # nobody sees draft 2, draft 2 sees the context alone
    mask = mask.to(DEV)
    want = kvc.attend_tree(gk, gv, q, mask=mask, first=first)
    for lay in (gk, gv):
        for s in range(B * H):
            a = lay.slot_layout(s)
            b = s // H
            row = lay.store[a["payload_offset"]:a["payload_offset"] + (S + 40) * a["row_bytes"]].view(S + 40, -1)
            side = lay.store[a["side_offset"]:a["side_offset"] + (S + 40) * 2].view(torch.float16)
            for sl in (slice(0, int(first[b])), slice(S - N + 2, S - N + 3), slice(S, S + 40)):
                row[sl] = 0xFF
                side[sl] = float("inf")
                side[sl][::2] = float("nan")
    got = kvc.attend_tree(gk, gv, q, mask=mask, first=first)
    assert torch.equal(got, want) and bool(torch.isfinite(got).all())


def test_strides_and_shared_mask(kvc):
    """Queries as views of [B, N, Hq, D], the output written into such a view,
    one mask for the whole batch, a uint8 mask, untouched rows around the output."""
    B, H, rep, D, S, N = 2, 2, 3, 64, 333, 6
    gk, gv, rk, rv = make_layers(kvc, "uniform", "int8", B, H, D, S, 41, dev=DEV)
    q = torch.randn(B, N, H * rep, D, generator=torch.Generator().manual_seed(2))
    mask = random_tree(np.random.default_rng(2), 1, N)
    buf = torch.full((B, N + 2, H * rep, D + 8), 7.0, dtype=torch.float16, device=DEV)
    view = buf[:, 1:N + 1, :, :D].transpose(1, 2)
    kvc.attend_tree(gk, gv, q.to(DEV).transpose(1, 2), mask=_dev(mask[0]).to(torch.uint8) * 3, out=view)
    ref = reference(gk, rk, gv, rv, q.transpose(1, 2).double().numpy(), 1 / math.sqrt(D), N,
                    mask=np.repeat(mask, B, 0))
    check(view, ref)
    assert bool((buf[:, 0] == 7).all()) and bool((buf[:, -1] == 7).all()) and bool((buf[..., D:] == 7).all())


def test_repeated_and_on_a_stream(kvc):
    """The same call twice, on another stream and in a replayed graph: the same bits."""
    gk, gv, rk, rv = make_layers(kvc, "codebook", "int8", 1, 2, 128, 3000, 51, dev=DEV)
    q = _q(1, 8, 6, 128, 6).to(DEV)
    a = kvc.attend_tree(gk, gv, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = kvc.attend_tree(gk, gv, q, stream=s)
    s.synchronize()
    ws = torch.empty(kvc.attend_tree_workspace_bytes(gk, gv, 8, 6), dtype=torch.uint8, device=DEV)
    out = torch.zeros_like(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.attend_tree(gk, gv, q, out=out, workspace=ws)
    q2 = q.clone()
    q.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    half = out.clone()
    q.copy_(q2)
    ws.fill_(0xFF)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, out) and not torch.equal(a, half)
    check(a, reference(gk, rk, gv, rv, q2.double().cpu().numpy(), 1 / math.sqrt(128), 6))


def test_layers_of_two_sizes_on_two_threads(kvc):
    """Two host threads call the same kernel with different amounts of shared
    memory in turn: what one thread asks for does not undo what the other did."""
    args = []
    for D, seed in ((128, 81), (32, 82)):
        gk, gv, _, _ = make_layers(kvc, "uniform", "int8", 1, 2, D, 200, seed, dev=DEV)
        args.append((gk, gv, _q(1, 4, 4, D, seed).to(DEV)))
    want = [kvc.attend_tree(*a) for a in args]
    torch.cuda.synchronize()
    got = []

    def once(a):
        t = threading.Thread(target=lambda: got.append(kvc.attend_tree(*a)))
        t.start()
        t.join()

    with concurrent.futures.ThreadPoolExecutor(1) as first:  # a thread that lives on
        got.append(first.submit(kvc.attend_tree, *args[0]).result())
        once(args[1])
        got.append(first.submit(kvc.attend_tree, *args[0]).result())
    torch.cuda.synchronize()
    assert len(got) == 3 and all(torch.equal(a, want[i]) for a, i in zip(got, (0, 1, 0)))


def test_extreme_queries(kvc):
    """Query rows of very different sizes in one call: each is right, and a row of
    NaN or infinities stays within its own row."""
    B, H, rep, D, S, N = 1, 1, 2, 128, 300, 4
    for kmode in ("codebook", "uniform"):
        gk, gv, rk, rv = make_layers(kvc, kmode, "int8", B, H, D, S, 61, dev=DEV)
        q = _q(B, rep, N, D, 7)
        q[0, 0, 1] *= 1e-4
        q[0, 1, 2] *= 1e3
        ref = reference(gk, rk, gv, rv, q.double().numpy(), 1 / math.sqrt(D), N)
        check(kvc.attend_tree(gk, gv, q.to(DEV)), ref)
        bad = q.clone()
        bad[0, 0, 0] = float("nan")
        bad[0, 1, 3] = float("inf")
        o = kvc.attend_tree(gk, gv, bad.to(DEV))
        del ref[0, 0], ref[0, 1]
        good = kvc.attend_tree(gk, gv, q.to(DEV))
        for x, i in ((0, 1), (0, 2), (0, 3), (1, 0), (1, 1)):
            assert torch.equal(o[0, x, i], good[0, x, i])
        assert not bool(torch.isfinite(o[0, 0, 0]).any()) and not bool(torch.isfinite(o[0, 1, 3]).any())


def test_refusals(kvc):
    B, H, D, S, N = 1, 2, 64, 40, 4
    gk, gv, _, _ = make_layers(kvc, "codebook", "int8", B, H, D, S, 71, capacity=S + 4, dev=DEV)
    q = _q(B, 2 * H, N, D, 8).to(DEV)

    def refused(status=-1, keys=gk, values=gv, q=q, **kw):
        with pytest.raises(kvc.KvcError) as e:
            kvc.attend_tree(keys, values, q, **kw)
        assert e.value.status == status

    refused(q=_q(B, 3, N, D, 8).to(DEV))                    # Hq not a multiple of H
    refused(q=_q(B, 2 * H, S + 1, D, 8).to(DEV))            # more drafts than tokens
    refused(keys=gv)                                        # int8 keys
    refused(values=gk)                                      # codebook values
    refused(scale=float("nan"))
    refused(scale=-1.0)
    refused(q=q.cpu())                                      # host memory
    refused(mask=torch.ones(N, N, dtype=torch.bool))
    refused(first=torch.zeros(B, dtype=torch.int32))
    refused(workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    refused(out=torch.empty(1, 1, 1, D, dtype=torch.float16, device=DEV).expand(B, 2 * H, N, D))
    flat = torch.empty(4 * H * N * D, dtype=torch.float16, device=DEV)
    refused(out=flat.as_strided((B, 2 * H, N, D), (0, D, D, 1)))                # heads and drafts meet
    refused(out=flat.as_strided((B, 2 * H, N, D), (0, (N - 1) * D, D, 1)))      # the last and the first draft
    gk.append(torch.randn(B, H, 1, D, device=DEV).half())
    refused()                                               # different lengths
    gk.trim(1)
    for bad in (dict(q=q[..., ::2]), dict(q=q[0]), dict(q=q.int()), dict(mask=torch.ones(N, N + 1, device=DEV)),
                dict(mask=torch.ones(2, N, N, dtype=torch.bool, device=DEV)),
                dict(mask=torch.ones(N, 2 * N, dtype=torch.bool, device=DEV)[:, ::2]),
                dict(first=torch.zeros(B, dtype=torch.int64, device=DEV)),
                dict(out=torch.empty(B, 2 * H, N, D, device=DEV))):
        with pytest.raises(ValueError):
            kvc.attend_tree(gk, gv, bad.pop("q", q), **bad)
    check_fine = kvc.attend_tree(gk, gv, q)
    assert bool(torch.isfinite(check_fine).all())


@pytest.mark.slow
def test_serving_sizes_sampled(kvc):
    """A long sequence split over many CTAs and a batch of several runs per CTA,
    some (batch, head) pairs checked."""
    _run(kvc, "codebook", "int8", 1, 4, 4, 128, 40001, 5, pairs={(0, 0), (0, 15)})
    _run(kvc, "uniform", "uniform", 16, 12, 1, 64, 1500, 17, dt="bf16", pairs={(0, 0), (7, 3), (15, 11)})
