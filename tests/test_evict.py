"""Accumulated attention weight and eviction on the GPU against their 64-bit
definitions.

Tolerance of a weight exp(s - lse), u = 2^-24: the score s is off by the fp32
summation, 2 D u sum|q||k| |scale| (one whole step per addition), and by the
roundings of the scaled value, the scale and the lse, 8 u (sum|q||k| |scale|
+ |lse|); exp2's approximation adds 2^-20, relative.  A score is a sum of
such weights and the old score: R more roundings of u.  Eviction moves bytes
and is compared exactly."""
import numpy as np
import pytest

import cache_ref as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def svp():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import spec_verify_paged_gb300 as m
    return m


def _io(dtype):
    return None if dtype == "f32" else "bf16"


def _cache_io(dtype):
    return "bf16" if dtype == "bf16" else None


SCORES = [
    # dtype, d, hq, hkv, q_len, lens, mask, k_scale
    ("bf16", 128, 4, 4, 1, [1, 15, 16, 17, 200], {}, 1.0),
    ("bf16", 64, 12, 4, 3, [3, 20, 150], {}, 1.0),
    ("bf16", 128, 32, 2, 9, [9, 100], {}, 1.0),             # 144 rows: two launches
    ("fp4", 128, 32, 8, 5, [5, 64, 300], {}, 0.4),
    ("fp4", 64, 4, 4, 1, [1, 33, 90], {}, 1.0),
    ("fp8", 128, 8, 2, 2, [2, 47, 300], {}, 0.0371),
    ("fp8", 64, 6, 2, 4, [4, 64], {}, 1.0),
    ("f32", 64, 4, 2, 2, [2, 16, 60], {}, 1.0),
    ("f32", 128, 8, 1, 16, [16, 40], {}, 1.0),              # 128 fp32 rows
    ("bf16", 128, 8, 2, 4, [4, 40, 300], dict(n_sink=4, window=37), 1.0),
    ("fp4", 128, 4, 4, 1, [1, 40, 300], dict(n_sink=20, window=1), 1.0),
    ("fp4", 128, 16, 4, 15, [15, 40, 300], "tree", 1.0),
    ("f32", 64, 2, 2, 6, [6, 40], "tree", 1.0),
    ("fp4", 128, 32, 2, 16, [16, 150], "tree", 1.0),        # 256 rows: two launches
    ("fp8", 128, 40, 2, 7, [7, 60], dict(n_sink=3, window=5), 1.0),  # 140 rows
]


@pytest.mark.parametrize("case", SCORES, ids=[str(i) for i in range(len(SCORES))])
def test_score_update(svp, case):
    import torch
    dtype, d, hq, hkv, ql, lens, mask, ks = case
    rng = np.random.default_rng(hq + ql + d)
    lens = np.asarray(lens, np.int32)
    table, total, _ = R.pages(rng, lens, spare=2)
    kc = R.make_cache(rng, dtype, total, hkv, d, ks, lens, table)
    q = rng.standard_normal((len(lens), ql, hq, d))
    q = q.astype(np.float32).astype(np.float64) if dtype == "f32" else R.bf16(q)
    scale = float(np.float32(1 / np.sqrt(d)))
    tree = np.tile(R.binary_tree(ql), (len(lens), 1)) if mask == "tree" else None
    m = {} if mask == "tree" else mask
    with np.errstate(invalid="ignore"):
        k = R.values(kc, dtype, d, float(np.float32(ks)))
    _, lse, mag, _ = R.attention(q, k, k, scale, lens, table, tree=tree, **m)
    lse = lse.astype(np.float32)
    old = rng.random((total, hkv, 16)).astype(np.float32)
    old[0, 0, :] = 0.0
    scores = R.to_gpu(old)
    got = svp.paged_score_update(
        R.to_gpu(q.astype(np.float32), _io(dtype)), R.to_gpu(kc, _cache_io(dtype)),
        R.to_gpu(lse), R.to_gpu(table), R.to_gpu(lens), scores, scale=scale,
        k_scale=ks, tree_mask=None if tree is None else R.to_gpu(tree), **m)
    assert got is scores and svp.read_device_status() == 0
    ref, added = R.score_update(q, k, lse.astype(np.float64), scale, lens, table,
                                old, ql, tree=tree, **m)
    spread = (2 * d + 8) * U * mag.max() + 8 * U * (mag.max() + np.abs(lse).max())
    rows = ql * hq // hkv
    tol = added * (2 * spread + 2.0 ** -20 + rows * U) + np.abs(ref) * rows * U
    err = np.abs(scores.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()
    # rows no sequence holds keep their bits
    free = np.ones((total, 16), bool)
    for b, L in enumerate(lens):
        for j in range(L):
            free[table[b, j // 16], j % 16] = False
    kept = scores.cpu().numpy().transpose(0, 2, 1)[free]
    assert np.array_equal(kept, old.transpose(0, 2, 1)[free])


def test_score_fresh_rows_and_skipped_rows(svp):
    """n_fresh below q_len adds to what the older new rows had; a row whose
    lse is -inf adds nothing; weights of one row sum to one."""
    import torch
    rng = np.random.default_rng(3)
    d, hq, hkv, ql = 64, 2, 2, 3
    lens = np.array([40], np.int32)
    table, total, _ = R.pages(rng, lens)
    kc = R.make_cache(rng, "bf16", total, hkv, d)
    q = R.bf16(rng.standard_normal((1, ql, hq, d)))
    args = [R.to_gpu(q, "bf16"), R.to_gpu(kc, "bf16")]
    pg = [R.to_gpu(table), R.to_gpu(lens)]
    _, lse = svp.paged_decode_attention(args[0], args[1], args[1], *pg)
    lse[0, 1, 0] = -float("inf")
    scores = torch.full((total, hkv, 16), 2.0, device="cuda")
    svp.paged_score_update(*args, lse, *pg, scores, n_fresh=1)
    s = R.logical(scores.cpu().numpy()[..., None], table[0], 0, 40)[:, 0]
    t = R.logical(scores.cpu().numpy()[..., None], table[0], 1, 40)[:, 0]
    # head 0: rows 0 and 2 of three; head 1: all three; 39 old scores of 2
    assert abs(s.sum() - 78 - 2) < 1e-3 and abs(t.sum() - 78 - 3) < 1e-3
    assert s[39] <= 1 and s[38] >= 2


EVICT = [
    # dtype, d, hkv, lens, budget, n_sink, n_recent
    ("bf16", 128, 3, [0, 1, 16, 40, 41, 300], 40, 4, 8),
    ("fp4", 128, 2, [100, 257], 64, 0, 0),
    ("fp4", 64, 2, [100, 257, 5], 33, 2, 31),              # nothing to choose
    ("fp8", 64, 1, [90], 1, 0, 0),
    ("fp8", 128, 2, [77, 200], 50, 50, 0),                 # sinks only
    ("f32", 64, 2, [70, 500], 61, 3, 7),
    ("f32", 128, 1, [128, 129], 128, 0, 128),
    ("bf16", 64, 2, [5000, 4097], 4000, 4, 64),            # two CTAs a group
    ("fp4", 128, 1, [33000], 1000, 4, 100),                # eight
    ("bf16", 128, 2, [3000, 900, 2999], 2999, 0, 0),       # one row goes
    ("fp8", 64, 3, [700, 0, 17], 16, 16, 0),
]


def _evict_inputs(dtype, d, hkv, lens, budget, seed=0, ties=True):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    need = -(-budget // 16)
    table, total, spare = R.pages(rng, lens, spare=need * len(lens) + 3)
    kc, vc = (R.make_cache(rng, dtype, total, hkv, d) for _ in range(2))
    s = rng.random((total, hkv, 16)).astype(np.float32)
    if ties:
        s = np.where(rng.random(s.shape) < 0.5, np.round(s * 4) / 4, s).astype(np.float32)
    dst = spare[:need * len(lens)].reshape(len(lens), need).copy()
    return kc, vc, s, table, lens, dst


def _apply(caches, kept, table, dst):
    """The caches and scores after the kept rows have moved (numpy)."""
    out = [c.copy() for c in caches]
    for b in range(kept.shape[0]):
        for h in range(kept.shape[1]):
            pos = kept[b, h][kept[b, h] >= 0]
            slot = np.arange(len(pos))
            for o, c in zip(out, caches):
                o[dst[b, slot // 16], h, slot % 16] = c[table[b, pos // 16], h, pos % 16]
    return out


def _raw(t):
    import torch
    if t.dtype == torch.bfloat16:
        return t.float().cpu().numpy()
    return t.cpu().numpy()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", EVICT, ids=[str(i) for i in range(len(EVICT))])
def test_evict(svp, case, in_place):
    dtype, d, hkv, lens, budget, n_sink, n_recent = case
    kc, vc, s, table, lens, dst = _evict_inputs(dtype, d, hkv, lens, budget)
    if table.shape[1] * 16 < budget:
        pytest.skip("the table cannot hold the budget in place")
    g = [R.to_gpu(kc, _cache_io(dtype)), R.to_gpu(vc, _cache_io(dtype)), R.to_gpu(s)]
    kept, new = svp.kv_evict(*g, R.to_gpu(table), R.to_gpu(lens), budget, n_sink,
                             n_recent, None if in_place else R.to_gpu(dst))
    assert svp.read_device_status() == 0
    ref, ref_lens = R.evict(s, lens, table, budget, n_sink, n_recent, hkv)
    assert np.array_equal(kept.cpu().numpy(), ref)
    assert np.array_equal(new.cpu().numpy(), ref_lens)
    for got, want in zip(g, _apply([kc, vc, s], ref, table, table if in_place else dst)):
        assert np.array_equal(_raw(got), want)


def test_evict_in_place_through_an_equal_table(svp):
    """A destination table that repeats the first entries of the block table
    is the in-place move, and new_lens may be seq_lens itself."""
    import torch
    kc, vc, s, table, lens, _ = _evict_inputs("bf16", 128, 2, [900, 300], 250)
    g = [R.to_gpu(kc, "bf16"), R.to_gpu(vc, "bf16"), R.to_gpu(s)]
    gl = R.to_gpu(lens)
    kept, new = svp.kv_evict(*g, R.to_gpu(table), gl, 250, 4, 16,
                             R.to_gpu(table[:, :16].copy()), new_lens=gl)
    assert new is gl
    ref, ref_lens = R.evict(s, lens, table, 250, 4, 16, 2)
    assert np.array_equal(kept.cpu().numpy(), ref)
    assert np.array_equal(gl.cpu().numpy(), ref_lens)
    for got, want in zip(g, _apply([kc, vc, s], ref, table, table)):
        assert np.array_equal(_raw(got), want)


def test_evict_leaves_shared_prefixes_intact(svp):
    """Three sequences share pages; their kept rows go to pages of their own
    and nothing else changes."""
    kc, vc, s, table, lens, dst = _evict_inputs("fp4", 128, 2, [300, 260, 90], 60)
    table[1, :10] = table[0, :10]
    table[2, :5] = table[0, :5]
    g = [R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(s)]
    kept, new = svp.kv_evict(*g, R.to_gpu(table), R.to_gpu(lens), 60, 2, 10, R.to_gpu(dst))
    ref, ref_lens = R.evict(s, lens, table, 60, 2, 10, 2)
    assert np.array_equal(kept.cpu().numpy(), ref)
    assert np.array_equal(new.cpu().numpy(), ref_lens)
    for got, want in zip(g, _apply([kc, vc, s], ref, table, dst)):
        assert np.array_equal(_raw(got), want)


def test_two_evictions_at_once_and_replayed(svp):
    """Two streams evict different sequences of one cache at the same time;
    a captured eviction replayed on restored caches gives the same bytes."""
    import torch
    kc, vc, s, table, lens, dst = _evict_inputs("bf16", 128, 2, [1500, 1400, 900], 400)
    first = [R.to_gpu(kc, "bf16"), R.to_gpu(vc, "bf16"), R.to_gpu(s)]
    gt, gl = R.to_gpu(table), R.to_gpu(lens)
    kept, new = svp.kv_evict(*first, gt, gl, 400, 4, 16)
    g = [R.to_gpu(kc, "bf16"), R.to_gpu(vc, "bf16"), R.to_gpu(s)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    parts = []
    for st, rows in zip(streams, (slice(0, 1), slice(1, 3))):
        with torch.cuda.stream(st):
            parts.append(svp.kv_evict(*g, gt[rows].contiguous(), gl[rows].contiguous(),
                                      400, 4, 16))
    torch.cuda.synchronize()
    assert torch.equal(torch.cat([p[0] for p in parts]), kept)
    for a, b in zip(g, first):
        assert torch.equal(a, b)
    start = [R.to_gpu(kc, "bf16"), R.to_gpu(vc, "bf16"), R.to_gpu(s)]
    for t, x in zip(g, start):
        t.copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k2, n2 = svp.kv_evict(*g, gt, gl, 400, 4, 16)
    for _ in range(2):
        for t, x in zip(g, start):
            t.copy_(x)
        k2.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(k2, kept) and torch.equal(n2, new)
        for a, b in zip(g, first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["zero", "signs", "nan", "inf", "equal", "tiny"])
def test_evict_score_orders(svp, kind):
    """Equal scores (lowest position first), both zeros, NaN and infinities,
    negative and subnormal scores."""
    kc, vc, s, table, lens, dst = _evict_inputs("fp8", 64, 2, [200, 70], 48)
    rng = np.random.default_rng(1)
    pick = rng.random(s.shape)
    if kind == "zero":
        s[:] = np.where(pick < 0.5, 0.0, -0.0)
    elif kind == "signs":
        s[:] = s - 0.5
    elif kind == "nan":
        s[:] = np.where(pick < 0.9, np.nan, np.where(pick < 0.95, -np.inf, s))
    elif kind == "inf":
        s[:] = np.where(pick < 0.5, np.inf, np.where(pick < 0.8, -np.inf, s))
    elif kind == "equal":
        s[:] = 0.75
    else:
        s[:] = np.float32(1e-45) * np.round(pick * 5)
    g = [R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(s)]
    kept, _ = svp.kv_evict(*g, R.to_gpu(table), R.to_gpu(lens), 48, 2, 5, R.to_gpu(dst))
    ref, _ = R.evict(s, lens, table, 48, 2, 5, 2)
    assert np.array_equal(kept.cpu().numpy(), ref)


def test_evict_beyond_the_key_cache(svp):
    """More positions per CTA than shared memory holds keys of."""
    import torch
    L, budget = 8 * 16384 + 1000, 5000
    rng = np.random.default_rng(2)
    lens = np.array([L], np.int32)
    need = -(-budget // 16)
    table, total, spare = R.pages(rng, lens, spare=need)
    s = rng.random((total, 1, 16)).astype(np.float32)
    s = np.where(rng.random(s.shape) < 0.3, np.float32(0.5), s)
    kc = torch.arange(total * 16, device="cuda").to(torch.float32).view(total, 1, 16, 1)
    kc = kc.expand(-1, -1, -1, 64).contiguous()
    vc = -kc
    kept, new = svp.kv_evict(kc, vc, R.to_gpu(s), R.to_gpu(table), R.to_gpu(lens),
                             budget, 3, 700, R.to_gpu(spare[:need][None].copy()))
    ref, ref_lens = R.evict(s, lens, table, budget, 3, 700, 1)
    assert np.array_equal(kept.cpu().numpy(), ref) and int(new[0]) == budget
    pos = ref[0, 0]
    want = table[0, pos // 16].astype(np.int64) * 16 + pos % 16
    slot = np.arange(budget)
    got = kc.cpu().numpy()[spare[slot // 16], 0, slot % 16, 5]
    assert np.array_equal(got, want.astype(np.float32))


def test_evict_bad_pages_and_lengths(svp):
    kc, vc, s, table, lens, dst = _evict_inputs("bf16", 64, 1, [100, 90, 60], 50)
    bad_lens = lens.copy()
    bad_lens[1] = 10 ** 6
    bad = table.copy()
    bad[0, 2] = -5
    g = [R.to_gpu(kc, "bf16"), R.to_gpu(vc, "bf16"), R.to_gpu(s)]
    kept, new = svp.kv_evict(*g, R.to_gpu(bad), R.to_gpu(bad_lens), 50, 0, 0, R.to_gpu(dst))
    assert svp.read_device_status() == 3
    assert new.tolist() == [50, -1, 50] and (kept[1] == -1).all()
    low = s.copy()
    low[table[0, 2]] = -np.inf
    ref, _ = R.evict(low, lens, table, 50, 0, 0, 1)
    assert np.array_equal(kept[[0, 2]].cpu().numpy(), ref[[0, 2]])


def test_decode_with_eviction(svp):
    """The operators as they are used: steps of append, attention, score
    update, and an eviction in place whenever a sequence outgrows its budget,
    over a 4-bit cache -- against the 64-bit forms run on the same stored
    rows; then the same step captured into a graph and replayed."""
    import torch
    rng = np.random.default_rng(17)
    B, hq, hkv, d, budget, n_sink, n_recent = 2, 8, 2, 128, 64, 4, 16
    room = 96
    width = room // 16
    table = rng.permutation(B * width).astype(np.int32).reshape(B, width)
    lens = np.array([60, 20], np.int32)
    kc = R.quantise(R.bf16(rng.standard_normal((B * width, hkv, 16, d))), 1.0)
    vc = R.quantise(R.bf16(rng.standard_normal((B * width, hkv, 16, d))), 1.0)
    s = rng.random((B * width, hkv, 16)).astype(np.float32)
    gk, gv, gs, gt = (R.to_gpu(x) for x in (kc, vc, s, table))
    gl = R.to_gpu(lens)
    scale = float(np.float32(1 / np.sqrt(d)))

    def step(q, k, v):
        gl.add_(1)
        svp.kv_append(k, v, gk, gv, gt, gl)
        out, lse = svp.paged_decode_attention(q, gk, gv, gt, gl, scale=scale)
        svp.paged_score_update(q, gk, lse, gt, gl, gs, scale=scale)
        svp.kv_evict(gk, gv, gs, gt, gl, budget, n_sink, n_recent, new_lens=gl)
        return out, lse

    for it in range(8):
        q, k, v = (R.bf16(rng.standard_normal((B, 1, h, d))) for h in (hq, hkv, hkv))
        # the 64-bit forms on the rows the cache holds
        lens = lens + 1
        kc, vc, s = gk.cpu().numpy(), gv.cpu().numpy(), gs.cpu().numpy()
        for b in range(B):
            at = table[b, (lens[b] - 1) // 16], slice(None), (lens[b] - 1) % 16
            kc[at], vc[at] = R.quantise(k[b, 0], 1.0), R.quantise(v[b, 0], 1.0)
        kval, vval = R.values(kc, "fp4", d), R.values(vc, "fp4", d)
        o_ref, l_ref, mag, vmax = R.attention(q, kval, vval, scale, lens, table)
        s_ref, _ = R.score_update(q, kval, l_ref, scale, lens, table, s, 1)
        gpu = [R.to_gpu(x, "bf16") for x in (q, k, v)]
        if it == 5:   # the rest of the steps through a captured graph
            held = [t.clone() for t in gpu]
            graph = torch.cuda.CUDAGraph()
            state = [t.clone() for t in (gk, gv, gs, gl)]
            with torch.cuda.graph(graph):
                result = step(*held)
            for t, x in zip((gk, gv, gs, gl), state):
                t.copy_(x)
        if it < 5:
            out, lse = step(*gpu)
        else:
            for t, x in zip(held, gpu):
                t.copy_(x)
            graph.replay()
            out, lse = result
        spread = (2 * d + 16) * U * (mag.max() + np.abs(l_ref).max())
        assert np.abs(lse.cpu().numpy() - l_ref).max() <= 2 * spread + 2.0 ** -18
        err = np.abs(out.double().cpu().numpy() - o_ref)
        assert (err <= (2 * spread + 2.0 ** -11 + 2.0 ** -16) * vmax.max() +
                2.0 ** -8 * np.abs(o_ref)).all()
        # scores before the move decide the kept rows: compare those whose
        # order is clear of the weights' rounding through the moved scores
        kept, new = R.evict(s_ref.astype(np.float32), lens, table, budget, n_sink,
                            n_recent, hkv)
        lens = new
        assert np.array_equal(gl.cpu().numpy(), new)
        moved = _apply([s_ref], kept, table, table)[0]
        got = gs.double().cpu().numpy()
        for b in range(B):
            for h in range(hkv):
                a = R.logical(got[..., None], table[b], h, new[b])[:, 0]
                w = R.logical(moved[..., None], table[b], h, new[b])[:, 0]
                # summed weights: relative error of one step's weights, in all
                assert np.abs(a - w).max() <= 1e-4 * np.abs(w).max()
    assert svp.read_device_status() == 0
