"""Windowed attention and eviction in a cache whose value rows lie past 2^32 bytes."""
import numpy as np
import pytest
import torch

from kvc_cases import fit_codebook

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
D, S, TAIL = 128, 34_000_000, 4000


@pytest.fixture(scope="module")
def kvc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import rank_quantized_kv_gb300 as kvc

    kvc.load_library()
    return kvc


def _layers(kvc, capacity):
    pk = fit_codebook(D, 3)
    return (kvc.KVCacheLayer("codebook", 1, 1, D, in_dtype="f16", capacity=capacity, device=DEV, **pk),
            kvc.KVCacheLayer("int8", 1, 1, D, in_dtype="f16", capacity=capacity, device=DEV))


def test_offsets_past_32_bits(kvc):
    """The last rows seen through a window equal those of a short cache of the sinks and
    the same last rows: either is off by half a step of fp16 and fp32 sums, 2^-11 of the
    largest value and little more, so that 2^-9 holds both; weights by fp32's sums of at
    most 48 + 128 products and the exponential, 2^-15 of a score of at most 16 each."""
    assert S * D > 1 << 32
    gen = torch.Generator(device=DEV).manual_seed(5)
    bulk = torch.randn(1, 1, 1_000_000, D, generator=gen, device=DEV, dtype=torch.float16)
    tail = torch.randn(1, 1, TAIL, D, generator=gen, device=DEV, dtype=torch.float16)
    far, near, kept = _layers(kvc, S), _layers(kvc, TAIL + 4), _layers(kvc, 5000)
    for lay in far:
        left = S - TAIL
        while left:
            n = min(left, bulk.shape[2])
            lay.append(bulk[:, :, :n])
            left -= n
        lay.append(tail)
    for lay in near:
        lay.append(bulk[:, :, :4])
        lay.append(tail)
    q = torch.randn(1, 4, 2, D, generator=gen, device=DEV)
    for weights in (False, True):
        w = torch.zeros(1, 1, S, device=DEV) if weights else None
        v = torch.zeros(1, 1, TAIL + 4, device=DEV) if weights else None
        a = kvc.attend_window(*far, q, window=3000, sinks=4, weights=w)
        b = kvc.attend_window(*near, q, window=3000, sinks=4, weights=v)
        assert float((a.float() - b.float()).abs().max()) <= 2 ** -9 * float(b.float().abs().max())
    assert bool((w[0, 0, 4:S - TAIL] == 0).all())
    w = torch.cat([w[0, 0, :4], w[0, 0, S - TAIL:]])
    assert float((w - v[0, 0]).abs().max()) <= 2 * 2 * 16 * 2.0 ** -15 * float(v.max())
    # 1996 heavy tokens anywhere, the sinks and the last 3000
    heavy = np.random.default_rng(3).choice(np.arange(4, S - 3000), 1996, replace=False)
    w = torch.zeros(1, 1, S, device=DEV)
    w[0, 0, torch.from_numpy(heavy).to(DEV)] = 1.0
    index, _ = kvc.evict(*far, w, 5000, sinks=4, recent=3000, into=(*kept, None))
    want = np.concatenate([np.arange(4), np.sort(heavy), np.arange(S - 3000, S)])
    assert np.array_equal(index[0, 0].cpu().numpy(), want)
    for src, dst in zip(far, kept):
        for x, y in zip(src.slot_rows(0), dst.slot_rows(0)):
            assert torch.equal(x[index[0, 0].long()], y)
    # and in place
    kvc.evict(*far, w, 5000, sinks=4, recent=3000)
    for src, dst in zip(far, kept):
        assert len(src) == 5000
        for x, y in zip(src.slot_rows(0), dst.slot_rows(0)):
            assert torch.equal(x, y)
    assert bool((w[0, 0, 5000:] == 0).all()) and float(w.sum()) == 1996.0
