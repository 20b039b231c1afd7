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


# ------------------------------------- the last launch of a call of several

def _guarded(svp, q, kc, table, split_pages=0):
    """A workspace of exactly the size the call asks for, and the bytes behind
    it (0xa5)."""
    import ctypes
    import torch
    from spec_verify_paged_gb300 import binding as bd
    d = q.shape[-1]
    code = bd._cache_code(kc, q.dtype)
    dims = bd.SvpDims(q.shape[0], q.shape[2], kc.shape[1], d, 16, table.shape[1],
                      kc.shape[0], code, None, 0, split_pages, 0, 1.0, 1.0)
    need = svp.load_library().paged_decode_workspace_size(ctypes.byref(dims), q.shape[1], 0, 0)
    whole = torch.full((need + (64 << 20),), 0xa5, dtype=torch.uint8, device="cuda")
    return whole[:need], whole[need:]


def _torch_attention(q, k, v, scale):
    """q [.., H, D], k and v [.., n, H, D] of one row each, fp64."""
    x = (k.double() * q.double()[:, None]).sum(-1) * scale
    p = x.softmax(1)
    return (p[..., None] * v.double()).sum(1), x.logsumexp(1)


def test_last_launch_stays_in_the_workspace_bf16(svp):
    """4100 sequences on the CUDA cores: 4096 short ones, then a launch of
    four long ones, whose CTAs an SM holds more of."""
    import torch
    B, hkv, d, width = 4100, 2, 128, 600
    g = torch.Generator(device="cuda").manual_seed(3)
    pages = 1 + 4 * width
    kc, vc = (torch.randn((pages, hkv, 16, d), device="cuda", generator=g).bfloat16()
              for _ in range(2))
    q = torch.randn((B, 1, hkv, d), device="cuda", generator=g).bfloat16()
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    table[4096:] = torch.arange(1, pages, dtype=torch.int32, device="cuda").view(4, width)
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    lens[4096:] = 16 * width - torch.arange(4, dtype=torch.int32, device="cuda")
    ws, guard = _guarded(svp, q, kc, table)
    out, lse = svp.paged_decode_attention(q, kc, vc, table, lens, scale=0.1, workspace=ws)
    assert svp.read_device_status() == 0
    assert (guard == 0xa5).all()
    # rows of one key: the value itself and its score (128 products in fp32)
    assert torch.equal(out[:4096, 0], vc[0, :, 0].expand(4096, -1, -1))
    for b in range(4096, B):
        n = int(lens[b])
        k, v = (c[table[b].long()].transpose(1, 2).flatten(0, 1)[None, :n] for c in (kc, vc))
        o, l = _torch_attention(q[b], k, v, 0.1)
        # bf16 output, half a step, and fp32 sums of 9600 weights
        assert (out[b].double() - o).abs().max() <= 2.0 ** -8 * o.abs().max() + 1e-4
        assert (lse[b].double() - l).abs().max() <= 1e-4


def test_last_launch_stays_in_the_workspace_4bit(svp):
    """1018 sequences of a page each, 20 rows: the first launch takes units of
    24 rows, the last has fewer pages than those want, and slices of a size
    that one CTA's warps are the whole workspace."""
    import torch
    B, hkv, group, d, split = 1018, 48, 20, 64, 12289
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn((B, 1, hkv * group, d), device="cuda", generator=g).bfloat16()
    x = torch.randn((1, 16, hkv, d), device="cuda", generator=g).bfloat16()
    kc = torch.zeros((1, hkv, 16, svp.fp4_row_bytes(d)), dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), 16, dtype=torch.int32, device="cuda")
    svp.kv_append(x, x, kc, vc, table[:1], lens[:1])
    k, v = svp.kv_gather(kc, vc, table[:1], lens[:1], 16)
    ws, guard = _guarded(svp, q, kc, table, split)
    out, lse = svp.paged_decode_attention(q, kc, vc, table, lens, scale=0.1, workspace=ws,
                                          split_pages=split)
    assert svp.read_device_status() == 0
    assert (guard == 0xa5).all()
    qs = q[:, 0].unflatten(1, (hkv, group))
    for h in range(0, hkv, 7):
        s = torch.einsum("bgd,nd->bgn", qs[:, h].double(), k[0, :, h].double()) * 0.1
        o = torch.einsum("bgn,nd->bgd", s.softmax(-1), v[0, :, h].double())
        at = slice(h * group, (h + 1) * group)
        # fp16 weights (2^-11) of values up to max|v|, bf16 output
        tol = 2.0 ** -10 * v[0, :, h].abs().max() + 2.0 ** -8 * o.abs()
        assert ((out[:, 0, at].double() - o).abs() <= tol).all()
        assert (lse[:, 0, at].double() - s.logsumexp(-1)).abs().max() <= 1e-4


# ------------------------------------------------------- masks at their ends

@pytest.mark.parametrize("dtype", ["bf16", "fp4"])
def test_all_keys_are_sinks(svp, dtype):
    """n_sink up to INT_MAX beside a window: every key is visible, to attention
    and to the score update, as without a window."""
    import torch
    rng = np.random.default_rng(4)
    lens = np.array([1500, 3], np.int32)
    table, total, _ = R.pages(rng, lens, width=200)
    cache = [R.to_gpu(R.make_cache(rng, dtype, total, 2, 64), "bf16" if dtype == "bf16" else None)
             for _ in range(2)]
    q = R.to_gpu(R.bf16(rng.standard_normal((2, 2, 4, 64))), "bf16")
    pg = [R.to_gpu(table), R.to_gpu(lens)]
    want = svp.paged_decode_attention(q, *cache, *pg)
    for n_sink in (2 ** 31 - 16, 2 ** 31 - 1):
        for window in (1, 2 ** 31 - 1):
            m = dict(n_sink=n_sink, window=window)
            out, lse = svp.paged_decode_attention(q, *cache, *pg, **m)
            # the same slices of the same pages
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
            s = [torch.zeros((total, 2, 16), device="cuda") for _ in range(2)]
            svp.paged_score_update(q, cache[0], lse, *pg, s[0])
            svp.paged_score_update(q, cache[0], lse, *pg, s[1], **m)
            assert torch.equal(*s) and float(s[0].sum()) > 0
    assert svp.read_device_status() == 0


@pytest.mark.parametrize("path", [2, 3])
@pytest.mark.parametrize("hq", [2, 20, 30, 48])
def test_zero_query_rows_and_tiny_factors(svp, path, hq):
    """A query row of zeros weighs every visible key the same, however small
    scale * k_scale is."""
    import torch
    rng = np.random.default_rng(hq)
    d, ql, lens = 128, 2, np.array([2, 37, 130, 700], np.int32)
    table, total, _ = R.pages(rng, lens)
    kc = R.make_cache(rng, "fp4", total, 2, d, 1.0, lens, table)
    vc = R.make_cache(rng, "fp4", total, 2, d, 1.0, lens, table)
    q = R.bf16(rng.standard_normal((len(lens), ql, hq, d)))
    q[:, :, ::2] = 0
    out, lse = svp.paged_decode_attention(
        R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table),
        R.to_gpu(lens), scale=1.0, k_scale=1e-30, kernel_path=path)
    with np.errstate(invalid="ignore"):
        v = R.values(vc, "fp4", d)
    for b, L in enumerate(lens):
        for i in range(ql):
            n = L - ql + i + 1
            for h in range(hq):    # a score is below 1e-25: no weight differs
                vv = R.logical(v, table[b], h // (hq // 2), L)[:n]
                # fp16 weights, 2^-11; bf16 output, 2^-8
                tol = 2.0 ** -10 * np.abs(vv).max() + 2.0 ** -8 * np.abs(vv.mean(0))
                got = out[b, i, h].double().cpu().numpy()
                assert (np.abs(got - vv.mean(0)) <= tol).all()
                assert abs(float(lse[b, i, h]) - np.log(n)) <= 1e-5
    assert svp.read_device_status() == 0


@pytest.mark.parametrize("path", [2, 3])
@pytest.mark.parametrize("hq", [2, 20, 48])
@pytest.mark.parametrize("split", [0, 1])
def test_nan_query_rows_give_nan(svp, path, hq, split):
    """A row with a NaN is NaN, output and lse, in short sequences and in
    groups that many slices share; the other rows are as without it."""
    import torch
    rng = np.random.default_rng(hq)
    d, lens = 128, np.array([1, 90, 5000], np.int32)
    table, total, _ = R.pages(rng, lens)
    cache = [R.to_gpu(R.make_cache(rng, "fp4", total, 2, d, 1.0, lens, table))
             for _ in range(2)]
    q = R.to_gpu(R.bf16(rng.standard_normal((3, 1, hq, d))), "bf16")
    call = lambda x: svp.paged_decode_attention(
        x, *cache, R.to_gpu(table), R.to_gpu(lens), scale=0.1, kernel_path=path,
        split_pages=split)
    out, lse = call(q)
    bad = q.clone()
    row = hq // 2
    bad[:, 0, row, 5] = float("nan")
    o2, l2 = call(bad)
    assert torch.isnan(o2[:, 0, row]).all() and torch.isnan(l2[:, 0, row]).all()
    rest = [h for h in range(hq) if h != row]
    # (rows of a tile share the moves of its softmax reference: rounding)
    assert (o2[:, 0, rest].float() - out[:, 0, rest].float()).abs().max() <= 2.0 ** -6
    assert (l2[:, 0, rest] - lse[:, 0, rest]).abs().max() <= 1e-4
    assert svp.read_device_status() == 0


@pytest.mark.parametrize("dtype,paths", [("fp4", (2, 3)), ("bf16", (1, 3))])
def test_tables_of_2_to_the_27_pages(svp, dtype, paths):
    """A table whose width in tokens passes 32 bits: the same as a narrow one."""
    import torch
    rng = np.random.default_rng(6)
    d, lens = 128, np.array([50], np.int32)
    table, total, _ = R.pages(rng, lens)
    io = "bf16" if dtype == "bf16" else None
    wide = torch.full((1, 2 ** 27), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = R.to_gpu(table)
    x = R.to_gpu(R.bf16(rng.standard_normal((1, 2, 1, d))), "bf16")
    q = R.to_gpu(R.bf16(rng.standard_normal((1, 2, 4, d))), "bf16")
    gl = R.to_gpu(lens)
    start = R.make_cache(rng, dtype, total, 1, d)
    got = []
    for t in (R.to_gpu(table), wide):
        k, v = R.to_gpu(start, io), R.to_gpu(start, io)
        svp.kv_append(x, x, k, v, t, gl)
        res = [k, v, *svp.kv_gather(k, v, t, gl, 50)]
        for path in paths:
            out, lse = svp.paged_decode_attention(q, k, v, t, gl, kernel_path=path)
            res += [out, lse]
        s = torch.zeros((total, 1, 16), device="cuda")
        svp.paged_score_update(q, k, lse, t, gl, s)
        got.append(res + [s])
        assert svp.read_device_status() == 0
    # (slices differ with the width: partial sums in another order, bf16 out)
    for a, b in zip(*got):
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -7


# -------------------------------------------- scores over infinite keys

@pytest.mark.parametrize("dtype,d,hq,hkv,ql", [
    ("bf16", 128, 2, 2, 1), ("bf16", 64, 6, 2, 1), ("bf16", 128, 6, 2, 3),
    ("bf16", 64, 8, 1, 1), ("bf16", 128, 32, 2, 9), ("f32", 64, 2, 2, 1),
])
def test_score_update_over_infinite_keys(svp, dtype, d, hq, hkv, ql):
    """A visible key with an infinite element: its score is -inf for every
    row, its weight 0, and its old score stays; the number of rows makes no
    difference."""
    import torch
    rng = np.random.default_rng(hq)
    lens = np.array([60], np.int32)
    table, total, _ = R.pages(rng, lens)
    io = "bf16" if dtype == "bf16" else None
    kc = R.make_cache(rng, dtype, total, hkv, d)
    q = R.bf16(rng.standard_normal((1, ql, hq, d)))
    q[..., 7] = -np.abs(q[..., 7]) - 1
    q = R.bf16(q)       # (what the call is given)
    for j in (3, 20, 47):
        kc[table[0, j // 16], :, j % 16, 7] = np.inf
    scale = float(np.float32(0.1))
    with np.errstate(invalid="ignore"):
        k = kc.astype(np.float64)
        _, lse, _, _ = R.attention(q, k, np.zeros_like(k), scale, lens, table)
    assert np.isfinite(lse).all()
    lse = lse.astype(np.float32)
    old = rng.random((total, hkv, 16)).astype(np.float32)
    scores = R.to_gpu(old)
    gq = R.to_gpu(q.astype(np.float32), io)
    svp.paged_score_update(gq, R.to_gpu(kc, io), R.to_gpu(lse), R.to_gpu(table),
                           R.to_gpu(lens), scores, scale=scale)
    ref, _ = R.score_update(q, k, lse.astype(np.float64), scale, lens, table, old, ql)
    assert np.isfinite(ref).all()
    got = scores.double().cpu().numpy()
    # a weight is off by a factor 1 + 2 (2 D + 8) u sum|q||k| scale at most (the
    # sum is about 10 at D = 128: 3e-4 if every rounding of the products' sum
    # fell the same way; 1e-4 is asked for)
    assert (np.abs(got - ref) <= 1e-4 * np.abs(ref)).all()
    for j in (3, 20, 47):
        at = table[0, j // 16], slice(None), j % 16
        assert np.array_equal(got[at], old[at].astype(np.float64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_left_out_by_their_lse(svp, dtype):
    """A row whose lse is -inf adds nothing, not even over a key whose score
    for it is +inf or NaN."""
    import torch
    rng = np.random.default_rng(2)
    d, hq, hkv, ql = 64, 4, 2, 2
    lens = np.array([40], np.int32)
    table, total, _ = R.pages(rng, lens)
    io = "bf16" if dtype == "bf16" else None
    kc = R.make_cache(rng, dtype, total, hkv, d)
    q = R.bf16(rng.standard_normal((1, ql, hq, d)))
    q[0, 0, 1, 7], q[0, 0, 3, 7] = 1.0, 0.0           # +inf and NaN scores
    q[0, 0, [0, 2], 7] = -1.0
    q[0, 1, :, 7] = -1.0
    kc[table[0, 0], :, 5, 7] = np.inf
    lse = rng.standard_normal((1, ql, hq)).astype(np.float32) + 4
    lse[0, 0, [1, 3]] = -np.inf
    old = rng.random((total, hkv, 16)).astype(np.float32)
    scores = R.to_gpu(old)
    scale = float(np.float32(0.125))
    svp.paged_score_update(R.to_gpu(q.astype(np.float32), io), R.to_gpu(kc, io),
                           R.to_gpu(lse), R.to_gpu(table), R.to_gpu(lens), scores,
                           scale=scale)
    ref, _ = R.score_update(q, kc.astype(np.float64), lse.astype(np.float64), scale,
                            lens, table, old, ql)
    assert np.isfinite(ref).all()
    got = scores.double().cpu().numpy()
    assert (np.abs(got - ref) <= 1e-4 * np.abs(ref)).all()
    at = table[0, 0], slice(None), 5
    assert np.array_equal(got[at], old[at].astype(np.float64))


# -------------------------------------- calls of different sizes, one process

SIZES = '''
import sys
import torch
import spec_verify_paged_gb300 as svp
kind, sizes = sys.argv[1], [int(x) for x in sys.argv[2].split(",")]
d, group = dict(tc4=(128, 40), tc=(128, 4), cores=(128, 1), mma=(64, 4))[kind]
most = max(sizes)
x = torch.randn((most, 1, 1, d), device="cuda").bfloat16()
q = torch.randn((most, 1, group, d), device="cuda").bfloat16()
row = svp.fp4_row_bytes(d) if kind == "tc4" else d
k = torch.zeros((most, 1, 16, row), device="cuda",
                dtype=torch.uint8 if kind == "tc4" else torch.bfloat16)
v = torch.zeros_like(k)
table = torch.arange(most, dtype=torch.int32, device="cuda").view(-1, 1)
lens = torch.ones(most, dtype=torch.int32, device="cuda")
svp.kv_append(x, x, k, v, table, lens)
want, _ = svp.kv_gather(k, v, table, lens, 1)
for n in sizes:
    out, lse = svp.paged_decode_attention(q[:n], k, v, table[:n], lens[:n])
    torch.cuda.synchronize()
    # one key a sequence: every row is its value
    assert torch.equal(out, want[:n].expand(-1, -1, group, -1)), n
    assert torch.isfinite(lse).all(), n
assert svp.read_device_status() == 0
print("done")
'''


@pytest.mark.parametrize("kind", ["tc4", "tc", "cores", "mma"])
@pytest.mark.parametrize("sizes", ["600,600", "300,10,300,600"])
def test_calls_of_changing_batch_sizes(svp, kind, sizes):
    """In a process of its own: a smaller launch leaves the next larger one
    its shared memory."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SIZES, kind, sizes], cwd=root,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------ flows of the README

def _score_inputs(seed, lens, hq, hkv, d, ql, table=None, total=None):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    if table is None:
        table, total, _ = R.pages(rng, lens)
    kc = R.make_cache(rng, "fp4", total, hkv, d)
    q = R.bf16(rng.standard_normal((len(lens), ql, hq, d)))
    old = rng.random((total, hkv, 16)).astype(np.float32)
    return q, kc, lens, table, old


def test_scores_of_shared_pages_one_call_a_sequence(svp):
    """Sequences that share pages are updated one after another: a shared
    page's scores hold what all of them gave it, and each evicts by that into
    pages of its own."""
    import torch
    rng = np.random.default_rng(21)
    lens = np.array([300, 260, 90], np.int32)
    hq, hkv, d, budget = 8, 2, 128, 60
    table, total, spare = R.pages(rng, lens, spare=3 * 4)
    table[1, :10] = table[0, :10]
    table[2, :5] = table[0, :5]
    q, kc, lens, table, old = _score_inputs(22, lens, hq, hkv, d, 1, table, total)
    scale = float(np.float32(0.1))
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(table), R.to_gpu(lens)]
    scores = R.to_gpu(old)
    _, lse = svp.paged_decode_attention(g[0], g[1], g[1], g[2], g[3], scale=scale)
    for b in range(3):
        at = slice(b, b + 1)
        svp.paged_score_update(g[0][at], g[1], lse[at], g[2][at], g[3][at], scores,
                               scale=scale)
    k = R.values(kc, "fp4", d)
    l64 = lse.double().cpu().numpy()
    ref = old
    for b in range(3):
        at = slice(b, b + 1)
        ref, _ = R.score_update(q[at], k, l64[at], scale, lens[at], table[at], ref, 1)
    got = scores.double().cpu().numpy()
    # weights within 2 (2 D + 8) 2^-24 sum|q||k| scale, which is below 13
    assert (np.abs(got - ref) <= 4e-4 * np.abs(ref)).all()
    dst = spare.reshape(3, 4)
    kept, new = svp.kv_evict(g[1], g[1].clone(), scores, g[2], g[3], budget, 2, 10,
                             R.to_gpu(dst))
    want, _ = R.evict(got.astype(np.float32), lens, table, budget, 2, 10, hkv)
    assert np.array_equal(kept.cpu().numpy(), want)


def test_scores_of_a_verification_leave_rejected_drafts_out(svp):
    """After a verification the rows of rejected drafts take an lse of -inf
    before the score update: the scores are those of the accepted rows alone,
    and the next step's rows start from zero where rejected ones stood."""
    import torch
    hq, hkv, d, ql = 8, 2, 128, 4
    q, kc, lens, table, old = _score_inputs(23, [64, 45, 90], hq, hkv, d, ql)
    scale = float(np.float32(0.1))
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(table), R.to_gpu(lens)]
    scores = R.to_gpu(old)
    _, lse = svp.paged_decode_attention(g[0], g[1], g[1], g[2], g[3], scale=scale)
    n_accepted = torch.tensor([0, 3, 1], dtype=torch.int32, device="cuda")
    rejected = torch.arange(ql, device="cuda") > n_accepted[:, None]
    lse.masked_fill_(rejected[..., None], -float("inf"))
    svp.paged_score_update(g[0], g[1], lse, g[2], g[3], scores, scale=scale)
    l64 = lse.double().cpu().numpy()
    k = R.values(kc, "fp4", d)
    ref = old
    for b, n in enumerate(n_accepted.tolist()):
        # the definition over the accepted rows of the shorter sequence
        at = slice(b, b + 1)
        short = lens[at] - ql + n + 1
        ref, _ = R.score_update(q[at, :n + 1], k, l64[at, :n + 1], scale, short,
                                table[at], ref, n + 1)
        for j in range(short[0], lens[b]):      # rejected: nobody sees them
            ref[table[b, j // 16], :, j % 16] = 0.0
    got = scores.double().cpu().numpy()
    assert (np.abs(got - ref) <= 4e-4 * np.abs(ref)).all()
    # the next step appends where the rejected rows were
    lens2 = lens - ql + n_accepted.cpu().numpy() + 1 + ql
    lens2 = np.minimum(lens2, 16 * np.array([(t >= 0).sum() for t in table])).astype(np.int32)
    gl = R.to_gpu(lens2)
    _, lse = svp.paged_decode_attention(g[0], g[1], g[1], g[2], gl, scale=scale)
    svp.paged_score_update(g[0], g[1], lse, g[2], gl, scores, scale=scale)
    ref, _ = R.score_update(q, k, lse.double().cpu().numpy(), scale, lens2, table, got, ql)
    assert (np.abs(scores.double().cpu().numpy() - ref) <= 4e-4 * np.abs(ref)).all()


# ---------------------------------------- the captured step over 4-bit caches

@pytest.mark.parametrize("hq,hkv,ql,lens,path,split,mask", [
    (8, 8, 1, [40, 900, 2100], 0, 0, {}),                   # slices
    (8, 2, 3, [3, 70, 1500], 2, 1, {}),                     # many slices
    (16, 2, 5, [17, 700, 1300], 2, 4, {}),                  # 40 rows, mma.sync
    (8, 2, 4, [300, 2000], 0, 2, dict(n_sink=5, window=300)),
    (16, 2, 5, [17, 700, 1300], 0, 0, {}),                  # 40 rows, tcgen05
    (8, 2, 3, [35, 500, 3000], 3, 0, {}),                   # 16-row units
    (32, 2, 2, [2, 33, 1100], 3, 8, {}),                    # 32-row units
    (32, 2, 4, [16, 129, 1100], 3, 0, dict(n_sink=3, window=200)),  # 64
    (8, 2, 16, [16, 33, 1600], 0, 0, "tree"),               # 64 rows
    (8, 2, 7, [7, 150, 1000], 2, 1, "tree"),
])
def test_step_runner_in_slices_and_on_tcgen05(svp, hq, hkv, ql, lens, path, split, mask):
    """The captured step, whose attention reads the prefix pages while the
    append runs, gives bit for bit what the single calls give, over groups
    that slices cut and over the tcgen05 kernel."""
    import torch
    rng = np.random.default_rng(hq + ql)
    d, vocab, B = 128, 64, len(lens)
    lens = np.asarray(lens, np.int32)
    steps = 4
    top = lens + steps * ql
    table, total, _ = R.pages(rng, top)
    start = [R.make_cache(rng, "fp4", total, hkv, d) for _ in range(2)]
    runs = [[R.to_gpu(x) for x in start] for _ in range(2)]
    kw = dict(split_pages=split, kernel_path=path, k_scale=0.4, v_scale=0.3)
    tree = mask == "tree"
    m = {} if tree else mask
    run = svp.StepRunner(*runs[0], B, hq, ql, table.shape[1], vocab=vocab if tree else 0,
                         tree_nodes=ql if tree else 0, **kw, **m)
    bits = np.tile(R.binary_tree(ql), (B, 1))
    gt = R.to_gpu(table)
    try:
        for step in range(steps):
            n = lens + step * ql
            t = [R.to_gpu(rng.standard_normal((B, ql, h, d)), "bf16") for h in (hq, hkv, hkv)]
            slot = step % 2
            for name, x in zip(("q", "k_new", "v_new"), t):
                run.host(slot, name)[:] = x.view(torch.int16).cpu().numpy().view(np.uint16)
            run.host(slot, "block_table")[:] = table
            run.host(slot, "seq_lens")[:] = n
            if tree:
                run.host(slot, "tree_mask")[:] = bits.view(np.uint32)
                run.host(slot, "parents")[:] = [(i - 1) // 2 if i else -1 for i in range(ql)]
                run.host(slot, "node_tokens")[:] = 1
                run.host(slot, "target_logits")[:] = 0
                run.host(slot, "draft_logits")[:] = 0
                run.host(slot, "uniforms")[:] = 0.5
            run.launch(slot)
            run.wait(slot)
            gl = R.to_gpu(n)
            svp.kv_append(t[1], t[2], *runs[1], gt, gl, k_scale=0.4, v_scale=0.3)
            if tree:
                out, lse = svp.paged_tree_attention(t[0], *runs[1], gt, gl, R.to_gpu(bits), **kw)
            else:
                out, lse = svp.paged_decode_attention(t[0], *runs[1], gt, gl, **kw, **m)
            got = torch.from_numpy(run.host(slot, "out").view(np.int16).copy())
            assert torch.equal(got, out.view(torch.int16).cpu())
            assert np.array_equal(run.host(slot, "lse"), lse.cpu().numpy())
            assert torch.isfinite(out.float()).all()
        for a, b in zip(*runs):
            assert torch.equal(a, b)
    finally:
        run.close()
    assert svp.read_device_status() == 0


@pytest.mark.parametrize("ql,mask", [(1, {}), (3, dict(n_sink=3, window=20)), (12, "tree")])
def test_more_sequences_than_a_tcgen05_launch_takes(svp, ql, mask):
    """600 sequences of 36 query rows on the automatic path: 512 and the rest,
    twice."""
    import torch
    rng = np.random.default_rng(ql)
    B, d, hq = 600, 128, 36 // ql
    lens = rng.integers(ql, 70, B).astype(np.int32)
    lens[[0, 511, 512, 599]] = (300, ql, 400, 17)
    table, total, _ = R.pages(rng, lens)
    kc = R.make_cache(rng, "fp4", total, 1, d, 1.0, lens, table)
    vc = R.make_cache(rng, "fp4", total, 1, d, 1.0, lens, table)
    q = R.bf16(rng.standard_normal((B, ql, hq, d)))
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table), R.to_gpu(lens)]
    if mask == "tree":
        mask = dict(tree=np.tile(R.binary_tree(ql), (B, 1)))
        call = lambda: svp.paged_tree_attention(*g, R.to_gpu(mask["tree"]), scale=0.1)
    else:
        call = lambda: svp.paged_decode_attention(*g, scale=0.1, **mask)
    out, lse = call()
    assert svp.read_device_status() == 0 and svp.last_launch_count() == 4
    again = call()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    with np.errstate(invalid="ignore"):
        k, v = (R.values(x, "fp4", d) for x in (kc, vc))
    o_ref, l_ref, mag, vmax = R.attention(q, k, v, float(np.float32(0.1)), lens, table, **mask)
    # as test_fp4_cache.py: fp32 sums of D products, fp16 weights, bf16 output
    u = 2.0 ** -24
    delta = 2 * d * u * mag + 8 * u * (mag + np.abs(l_ref))
    tol = ((2 * delta + 2.0 ** -11 + 2.0 ** -16) * vmax)[..., None] + 2.0 ** -8 * np.abs(o_ref)
    assert (np.abs(out.double().cpu().numpy() - o_ref) <= tol).all()
    err = np.abs(lse.double().cpu().numpy() - l_ref)
    assert (err <= 2 * delta + 2.0 ** -18 + 4 * u * np.abs(l_ref)).all()
