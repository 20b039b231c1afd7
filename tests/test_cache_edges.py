"""Calls on the edges of what the 4-bit cache, score and eviction entry points
document: tables far wider than the sequences, infinite keys, query rows that
are zero or NaN, launches of different sizes after one another, and the flows
the README shows for shared prefixes and rejected drafts.  On the GPU, against
the 64-bit forms of cache_ref.py."""
import numpy as np
import pytest

import cache_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def svp():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import spec_verify_paged_gb300 as m
    return m


# ----------------------------------------------- eviction out of wide tables

@pytest.mark.parametrize("width,lens,budget,n_sink,n_recent", [
    # two, four and eight CTAs a group, most of them without a position
    (300, [1, 2, 3, 5, 6, 7, 15, 17, 18, 19, 33, 300], 1, 0, 0),
    (600, [5, 21, 22, 23, 49, 50, 51, 390, 391], 4, 1, 1),
    (2048, [21, 37, 38, 39, 781, 782, 783, 785, 890, 897], 20, 2, 7),
    (2048, [700, 129, 131, 1000, 4097], 128, 4, 32),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_short_sequences_in_a_wide_table(svp, width, lens, budget, n_sink,
                                               n_recent, in_place):
    rng = np.random.default_rng(width + budget)
    lens = np.asarray(lens, np.int32)
    hkv, d, need = 2, 64, -(-budget // 16)
    table, total, spare = R.pages(rng, lens, spare=need * len(lens), width=width)
    kc, vc = (R.make_cache(rng, "fp4", total, hkv, d) for _ in range(2))
    s = rng.random((total, hkv, 16)).astype(np.float32)
    s = np.where(rng.random(s.shape) < 0.5, np.round(s * 4) / 4, s).astype(np.float32)
    dst = table if in_place else spare.reshape(len(lens), need)
    g = [R.to_gpu(x) for x in (kc, vc, s)]
    kept, new = svp.kv_evict(*g, R.to_gpu(table), R.to_gpu(lens), budget, n_sink,
                             n_recent, None if in_place else R.to_gpu(dst))
    assert svp.read_device_status() == 0
    ref, ref_lens = R.evict(s, lens, table, budget, n_sink, n_recent, hkv)
    assert np.array_equal(kept.cpu().numpy(), ref)
    assert np.array_equal(new.cpu().numpy(), ref_lens)
    for got, old in zip(g, (kc, vc, s)):
        want = old.copy()
        for b in range(len(lens)):
            for h in range(hkv):
                pos = ref[b, h][ref[b, h] >= 0]
                slot = np.arange(len(pos))
                want[dst[b, slot // 16], h, slot % 16] = old[table[b, pos // 16], h, pos % 16]
        assert np.array_equal(got.cpu().numpy(), want)
