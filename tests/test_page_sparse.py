"""Page bounds, page scores, page selection and attention over listed pages, on
the GPU, against the 64-bit forms of page_ref.py.

Tolerances.  Every sum of n products in fp32 is off by at most n + 2 roundings
of the sum of the magnitudes; the tensor cores add up to a step more in each,
so 2^-23 is counted for one.  A weight is rounded by 2^-8 (bf16) or 2^-11 (fp16)
of itself, an output by half a step of its type."""
import numpy as np
import pytest

import cache_ref as R
import page_ref as G

pytestmark = pytest.mark.gpu

DTYPES = ["f32", "bf16", "fp8", "fp4"]
SCALE = {"fp8": 2.0 ** -5, "fp4": 0.0371}


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


def _gpu_cache(x, dtype):
    return R.to_gpu(x, "bf16" if dtype == "bf16" else None)


def _f64(t):
    return t.float().double().cpu().numpy()


# ------------------------------------------------------------------ bounds

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 3)])
@pytest.mark.parametrize("n_new", [1, 16, 17, 40, None])
def test_bounds(svp, dtype, d, hkv, n_new):
    rng = np.random.default_rng(d + hkv + (n_new or 0))
    lens = np.array([0, 1, 15, 16, 17, 33, 100], np.int32)
    table, total, _ = R.pages(rng, lens, spare=3, width=9)
    k = R.make_cache(rng, dtype, total, hkv, d, SCALE.get(dtype, 1.0), lens, table)
    old = rng.integers(-3, 4, (total, hkv, 2, d)).astype(np.float64)
    b = R.to_gpu(old.astype(np.float32), "bf16")
    r = svp.kv_page_bounds(_gpu_cache(k, dtype), R.to_gpu(table), R.to_gpu(lens), b, n_new)
    assert r is b and svp.read_device_status() == 0
    want = G.bounds(R.values(k, dtype, d), lens, table, n_new or 10 ** 6, old)
    assert np.array_equal(_f64(b), want)  # rows past the lengths are NaN


def test_bounds_of_fp32_are_rounded_outward(svp):
    rng = np.random.default_rng(5)
    k = (rng.standard_normal((2, 1, 16, 64)) * np.exp(10 * rng.standard_normal((2, 1, 16, 64))))
    k = k.astype(np.float32)
    k[1] = np.abs(k[1])
    k[0, 0, :, 0] = 3.4e38    # rounds up to infinity
    k[0, 0, :, 1] = 1.0
    k[0, 0, :, 2] = -1.0 - 2.0 ** -20
    k[0, 0, :, 3] = -0.0
    table = np.array([[0, 1]], np.int32)
    b = R.to_gpu(np.zeros((2, 1, 2, 64), np.float32), "bf16")
    svp.kv_page_bounds(R.to_gpu(k), R.to_gpu(table), R.to_gpu(np.array([32], np.int32)), b)
    got = _f64(b)
    want = G.bounds(k.astype(np.float64), [32], table, 99, np.zeros((2, 1, 2, 64)))
    want[0, 0, 1, 0] = np.inf
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_bounds_nan_and_infinities(svp, dtype):
    rng = np.random.default_rng(6)
    lens, table = np.array([40], np.int32), np.array([[1, 0, 2]], np.int32)
    k = R.make_cache(rng, dtype, 3, 1, 64)
    if dtype == "fp4":
        k[1, 0, 3, 32] = 0xFF       # a NaN scale: 16 elements
        hurt = np.arange(16)
    elif dtype == "fp8":
        k[1, 0, 3, 5] = 0x7F
        hurt = np.array([5])
    else:
        k[1, 0, 3, 5] = np.nan
        k[0, 0, 0, 7] = -np.inf
        k[2, 0, 7, 9] = np.inf
        hurt = np.array([5])
    b = R.to_gpu(np.zeros((3, 1, 2, 64), np.float32), "bf16")
    svp.kv_page_bounds(_gpu_cache(k, dtype), R.to_gpu(table), R.to_gpu(lens), b)
    got = _f64(b)
    assert np.isnan(got[1, 0][:, hurt]).all()
    assert np.isnan(got).sum() == 2 * len(hurt)
    if dtype in ("f32", "bf16"):
        assert got[0, 0, 0, 7] == -np.inf and got[2, 0, 1, 9] == np.inf


def test_bounds_bad_data(svp):
    k = R.to_gpu(np.ones((3, 1, 16, 64), np.float32), "bf16")
    b = R.to_gpu(np.zeros((3, 1, 2, 64), np.float32), "bf16")
    t = np.array([[0, 3], [-1, 1], [0, 1], [0, 1]], np.int32)
    svp.kv_page_bounds(k, R.to_gpu(t), R.to_gpu(np.array([32, 32, -1, 33], np.int32)), b)
    assert svp.read_device_status() == 1 | 2
    assert _f64(b)[:2].min() == 1 and _f64(b)[2].max() == 0


# ------------------------------------------------------------------ scores

def _scores(svp, rng, dtype, d, hkv, group, ql, lens, scale, width=None):
    table, total, _ = R.pages(rng, lens, width=width)
    mid = rng.standard_normal((total, hkv, 1, d))
    bnd = R.bf16(np.concatenate([mid - 1.5, mid + 1.5], 2) *
                 np.where(rng.random((total, hkv, 1, d)) < 0.1, 5.0, 1.0))
    q = rng.standard_normal((len(lens), ql, hkv * group, d))
    q = q.astype(np.float32).astype(np.float64) if dtype == "f32" else R.bf16(q)
    got = svp.paged_page_scores(
        R.to_gpu(q.astype(np.float32), _io(dtype)), R.to_gpu(bnd.astype(np.float32), "bf16"),
        R.to_gpu(table), R.to_gpu(lens), scale=scale)
    return got, q, bnd, table


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,hkv,group,ql,scale", [
    (64, 1, 1, 1, 0.125), (128, 2, 4, 1, 0.0884), (128, 3, 3, 3, -0.2),
    (64, 2, 8, 5, 0.125), (128, 1, 8, 9, 0.1),
    (64, 2, 17, 8, 0.125),   # 136 rows: two launches of bf16, three of fp32
])
def test_scores(svp, dtype, d, hkv, group, ql, scale):
    rng = np.random.default_rng(d + group + ql)
    lens = np.array([0, 1, 16, 17, 250, 1000], np.int32)
    got, q, bnd, table = _scores(svp, rng, dtype, d, hkv, group, ql, lens, scale, 70)
    assert svp.read_device_status() == 0
    want, mag = G.scores(q, bnd, lens, table, np.float32(scale))
    got = _f64(got)
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    ok = np.isfinite(want)
    # 2 D terms (three parts of an fp32 q), and the product with the scale
    n = 2 * d * (3 if dtype == "f32" else 1) + 4
    assert (np.abs(got[ok] - want[ok]) <= n * 2.0 ** -23 * mag[ok]).all()


def test_scores_wide_table(svp):
    """Far more table than pages, many warps' tiles to a CTA."""
    rng = np.random.default_rng(9)
    lens = np.array([40000, 100, 16000, 7], np.int32)
    got, q, bnd, table = _scores(svp, rng, "bf16", 64, 2, 2, 1, lens, 0.125, 40001)
    b = bnd[np.maximum(table, 0)].transpose(0, 2, 1, 3, 4)   # [B, Hkv, W, 2, D]
    x = q[:, 0].reshape(4, 2, 2, 64)
    want = (np.einsum("bhgd,bhwd->bhgw", np.maximum(x, 0), b[:, :, :, 1]) +
            np.einsum("bhgd,bhwd->bhgw", np.minimum(x, 0), b[:, :, :, 0])).max(2) * 0.125
    there = (np.arange(40001) * 16 < lens[:, None])[:, None]
    got = _f64(got)
    assert np.isneginf(got[~np.broadcast_to(there, got.shape)]).all()
    err = np.abs(got - want)[np.broadcast_to(there, got.shape)]
    assert err.max() <= 132 * 2.0 ** -23 * 64 * 4 * 8 * 0.125


def test_scores_bound_the_attention_products(svp):
    """No scaled product of a row with a key of the page exceeds its score."""
    import torch
    rng = np.random.default_rng(11)
    lens = np.array([77, 160], np.int32)
    table, total, _ = R.pages(rng, lens)
    for dtype in DTYPES:
        ks = SCALE.get(dtype, 1.0)
        k = R.make_cache(rng, dtype, total, 2, 128, ks, lens, table)
        q = R.bf16(rng.standard_normal((2, 2, 8, 128)))
        b = torch.empty((total, 2, 2, 128), dtype=torch.bfloat16, device="cuda")
        t, n = R.to_gpu(table), R.to_gpu(lens)
        svp.kv_page_bounds(_gpu_cache(k, dtype), t, n, b)
        s = _f64(svp.paged_page_scores(R.to_gpu(q.astype(np.float32), _io(dtype)), b, t, n,
                                       scale=0.09, k_scale=ks))
        v = R.values(k, dtype, 128, ks)
        for i in range(2):
            for h in range(2):
                kk = R.logical(v, table[i], h, lens[i])
                x = np.einsum("qhd,nd->qhn", q[i, :, 4 * h:4 * h + 4], kk) * 0.09
                most = x.max((0, 1))
                tol = 300 * 2.0 ** -23 * (np.abs(kk).max() * 128 * 4 * 0.09)
                assert (most <= s[i, h][np.arange(len(kk)) // 16] + tol).all()


def test_scores_nan_infinities_and_bad_data(svp):
    rng = np.random.default_rng(12)
    lens = np.array([64, 64, 65, -2], np.int32)
    table = np.array([[0, 1, 2, 3], [4, 9, -1, 5], [0, 1, 2, 3], [0, 1, 2, 3]], np.int32)
    bnd = np.sort(rng.standard_normal((6, 1, 2, 64)), 2)
    bnd[1, 0, 1, 3] = np.inf
    bnd[2, 0, :, 5] = np.nan
    q = R.bf16(rng.standard_normal((4, 1, 1, 64)))
    q[0, 0, 0, 3] = 1.0          # 1 * inf + 0 * lo
    s = _f64(svp.paged_page_scores(
        R.to_gpu(q.astype(np.float32), "bf16"), R.to_gpu(bnd.astype(np.float32), "bf16"),
        R.to_gpu(table), R.to_gpu(lens), scale=0.5))
    assert svp.read_device_status() == 1 | 2
    assert np.isfinite(s[0, 0, [0, 3]]).all() and s[0, 0, 1] == np.inf and np.isnan(s[0, 0, 2])
    assert np.isfinite(s[1, 0, [0, 3]]).all() and np.isneginf(s[1, 0, [1, 2]]).all()
    assert np.isneginf(s[2:]).all()
    # a scale of zero: products of zero
    z = _f64(svp.paged_page_scores(
        R.to_gpu(q.astype(np.float32), "bf16"), R.to_gpu(bnd.astype(np.float32), "bf16"),
        R.to_gpu(table), R.to_gpu(np.array([16] * 4, np.int32)), scale=0.0))
    svp.read_device_status()
    assert (z[:, 0, 0] == 0).all()


# --------------------------------------------------------------- selection

@pytest.mark.parametrize("width,lens,n_select,n_sink,n_recent", [
    (1, [16, 0, 1], 1, 0, 1),
    (9, [1, 16, 17, 144, 130], 4, 1, 1),
    (9, [144, 130, 97], 4, 2, 2),           # nothing by score
    (200, [3200, 3199, 1000, 100], 17, 0, 0),
    (1000, [16000, 15985, 4000, 33], 100, 3, 8),
    (2048, [32768, 20000], 1024, 1, 4),
    (2049, [32784, 20000], 2000, 1, 4),
    (8192, [131072, 130001, 70000], 256, 1, 8),
    (16384, [262144, 250000], 300, 1, 8),
    (16385, [262145, 250000], 300, 1, 8),   # more than the registers hold
    (40000, [640000, 300000], 5000, 0, 1),
])
def test_select(svp, width, lens, n_select, n_sink, n_recent):
    rng = np.random.default_rng(width + n_select)
    lens = np.array(lens, np.int32)
    s = rng.standard_normal((len(lens), 3, width)).astype(np.float32)
    s[:, 1] = np.round(s[:, 1] * 2)         # ties by the hundred
    s[:, 2, ::3] = np.where(rng.random(s[:, 2, ::3].shape) < 0.2, np.nan, -np.inf)
    s[:, 2, 1::7] = np.inf
    got = svp.paged_select_pages(R.to_gpu(s), R.to_gpu(lens), n_select, n_sink, n_recent)
    assert svp.read_device_status() == 0
    want = G.select(s, lens, n_select, n_sink, n_recent)
    assert np.array_equal(got.cpu().numpy(), want)


def test_select_equal_scores_and_signs(svp):
    s = np.zeros((5, 1, 3000), np.float32)
    s[1] = -np.inf
    s[2] = np.nan
    s[3, 0, ::2] = -0.0                     # as +0
    s[4] = -np.nan
    lens = np.full(5, 48000, np.int32)
    got = svp.paged_select_pages(R.to_gpu(s), R.to_gpu(lens), 40, 2, 3).cpu().numpy()
    want = np.r_[np.arange(37), 2997:3000]
    assert (got == want).all()


def test_select_bad_lengths(svp):
    s = R.to_gpu(np.zeros((3, 2, 4), np.float32))
    got = svp.paged_select_pages(s, R.to_gpu(np.array([-1, 65, 64], np.int32)), 4)
    assert svp.read_device_status() == 2
    assert (got[:2] == -1).all() and got[2].tolist() == [[0, 1, 2, 3]] * 2


# ------------------------------------------------------- attention by list

def _lists(rng, lens, hkv, n_select, holes=True):
    """Lists in any order, with holes; the newest pages are among them."""
    out = np.full((len(lens), hkv, n_select), -1, np.int32)
    for b, L in enumerate(lens):
        n = -(-int(L) // 16)
        for h in range(hkv):
            k = min(n, n_select)
            take = rng.permutation(n)[:k]
            if holes and k > 3:
                take = take[:k - rng.integers(0, 2)]
            at = rng.permutation(n_select)[:len(take)]
            out[b, h, at] = take
            if holes and rng.random() < 0.3:
                out[b, h, out[b, h] < 0] = -rng.integers(1, 9)
    return out


def _sparse(svp, rng, dtype, d, hkv, group, ql, lens, n_select, split=0, tree=False,
            scale=None, lists=None, q=None, **kw):
    lens = np.array(lens, np.int32)
    table, total, _ = R.pages(rng, lens, spare=2)
    ks = SCALE.get(dtype, 1.0)
    vs = 0.75 * ks if dtype in SCALE else 1.0
    k, v = (R.make_cache(rng, dtype, total, hkv, d, x, lens, table) for x in (ks, vs))
    if q is None:
        q = rng.standard_normal((len(lens), ql, hkv * group, d))
    q = q.astype(np.float32).astype(np.float64) if dtype == "f32" else R.bf16(q)
    if lists is None:
        lists = _lists(rng, lens, hkv, n_select)
    bits = np.tile(R.binary_tree(ql), (len(lens), 1)) if tree else None
    scale = d ** -0.5 if scale is None else scale
    out, lse = svp.paged_sparse_attention(
        R.to_gpu(q.astype(np.float32), _io(dtype)), _gpu_cache(k, dtype),
        _gpu_cache(v, dtype), R.to_gpu(table), R.to_gpu(lens), R.to_gpu(lists),
        tree_mask=None if bits is None else R.to_gpu(bits), scale=scale,
        split_pages=split, k_scale=ks, v_scale=vs, **kw)
    ref = G.sparse_attention(q, R.values(k, dtype, d, ks), R.values(v, dtype, d, vs),
                             float(np.float32(scale)), lens, table, lists, bits)
    return out, lse, ref


def _check(dtype, d, out, lse, ref):
    want, wlse, mag, vmax = ref
    got, glse = _f64(out), lse.double().cpu().numpy()
    # the scores: D products, the scale's two roundings; in the exponent twice
    score = (d + 4) * 2.0 ** -23 * mag
    assert np.array_equal(np.isneginf(glse), np.isneginf(wlse))
    ok = np.isfinite(wlse)
    # 2^-20: the exponentials, their sum and the logarithm, and lse's own size
    assert (np.abs(glse[ok] - wlse[ok]) <=
            score[ok] + 2.0 ** -20 + 2.0 ** -23 * np.abs(wlse[ok])).all()
    weight = {"f32": 2.0 ** -20, "bf16": 2.0 ** -8, "fp8": 2.0 ** -11, "fp4": 2.0 ** -11}[dtype]
    # fp16 weights below 2^-20 of the largest are rounded by 2^-31 instead
    weight += 2.0 ** -19
    half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    tol = (weight + 2 * score) * vmax
    assert (np.abs(got - want) <= tol[..., None] + half * np.abs(want) + 1e-37).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,hkv,group,ql,n_select,split", [
    (64, 1, 1, 1, 1, 0),
    (128, 2, 1, 1, 9, 0),
    (128, 2, 4, 1, 12, 1),     # clusters of eight
    (64, 3, 5, 1, 12, 3),
    (128, 1, 4, 5, 12, 0),     # 20 rows: two row groups
    (64, 2, 7, 5, 20, 2),      # 35 rows
    (128, 1, 8, 8, 12, 4),     # 64 rows
    (128, 2, 5, 13, 12, 0),    # 65 rows: two units
    (64, 1, 33, 4, 5, 1),      # 132 rows
    (64, 2, 4, 3, 13, 0),      # 12 rows
    (128, 2, 8, 2, 13, 1),     # 16 rows, clusters
    (64, 1, 8, 3, 11, 2),      # 24 rows
])
def test_sparse(svp, dtype, d, hkv, group, ql, n_select, split):
    rng = np.random.default_rng(d + group + ql + n_select)
    lens = [ql, ql + 1, 16 * ((ql + 15) // 16), 33 + ql, 191, 192]
    out, lse, ref = _sparse(svp, rng, dtype, d, hkv, group, ql, lens, n_select, split)
    assert svp.read_device_status() == 0 and svp.last_launch_count() == 1
    _check(dtype, d, out, lse, ref)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,group,ql", [(64, 1, 2), (128, 4, 15), (128, 2, 16)])
def test_sparse_tree(svp, dtype, d, group, ql):
    rng = np.random.default_rng(d + group + ql)
    out, lse, ref = _sparse(svp, rng, dtype, d, 2, group, ql, [ql, 40, 47, 48, 130], 7,
                            tree=True)
    assert svp.read_device_status() == 0
    _check(dtype, d, out, lse, ref)


@pytest.mark.parametrize("dtype", DTYPES)
def test_sparse_long_lists(svp, dtype):
    """More entries than are looked up at once, with and without clusters; the
    same page many times, holes between."""
    rng = np.random.default_rng(21)
    lens = [300, 17]
    lists = rng.integers(-3, 19, (2, 2, 1500)).astype(np.int32)
    lists[1] = np.minimum(lists[1], 1)
    for split, d, group, ql in ((1500, 64, 2, 1), (0, 64, 2, 1), (1500, 128, 4, 3),
                                (0, 64, 7, 3)):
        out, lse, ref = _sparse(svp, rng, dtype, d, 2, group, ql, lens, 1500, split,
                                lists=lists)
        assert svp.read_device_status() == 0
        _check(dtype, d, out, lse, ref)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,hkv,group,ql,n_select,split", [
    (64, 2, 3, 2, 16, 1),     # an entry to a CTA
    (128, 1, 4, 5, 257, 0),   # 20 rows
    (128, 2, 7, 5, 300, 0),   # 35 rows
    (64, 1, 8, 1, 255, 0),    # one entry too few: clusters of eight
])
def test_sparse_clusters_of_sixteen(svp, dtype, d, hkv, group, ql, n_select, split):
    """Also with shares that list nothing, but one, and none at all."""
    rng = np.random.default_rng(d + ql + n_select)
    for kept in (slice(0, n_select), slice(n_select - 1, None), slice(3, 6), slice(0, 0)):
        lists = np.full((1, hkv, n_select), -1, np.int32)
        lists[..., kept] = rng.integers(0, 25, lists[..., kept].shape)
        out, lse, ref = _sparse(svp, rng, dtype, d, hkv, group, ql, [397], n_select, split,
                                lists=lists)
        assert svp.read_device_status() == 0
        _check(dtype, d, out, lse, ref)


@pytest.mark.parametrize("dtype", DTYPES)
def test_sparse_rows_that_see_nothing(svp, dtype):
    """Empty lists, and lists whose keys lie after a row's position."""
    rng = np.random.default_rng(22)
    lists = np.full((4, 1, 6), -1, np.int32)
    lists[1, 0, 3] = 2      # positions 32..: rows 0..3 of 35 - 5 do not see it
    lists[2, 0, :3] = [2, 1, 0]
    for split in (0, 1):
        out, lse, ref = _sparse(svp, rng, dtype, 128, 1, 3, 5, [35, 35, 35, 5], 6, split,
                                lists=lists)
        assert svp.read_device_status() == 0
        _check(dtype, 128, out, lse, ref)
        assert (_f64(out)[0] == 0).all() and np.isneginf(lse[0].cpu().numpy()).all()
        assert np.isneginf(lse[1, :2].cpu().numpy()).all()
        assert np.isfinite(lse[1, 2:].cpu().numpy()).all()


def test_sparse_over_all_pages_is_dense(svp):
    import torch
    rng = np.random.default_rng(23)
    lens = np.array([200, 75, 9], np.int32)
    table, total, _ = R.pages(rng, lens)
    k, v = (R.to_gpu(R.make_cache(rng, "bf16", total, 2, 128, lens=lens, table=table), "bf16")
            for _ in range(2))
    q = R.to_gpu(rng.standard_normal((3, 5, 8, 128)).astype(np.float32), "bf16")
    t, n = R.to_gpu(table), R.to_gpu(lens)
    pages = torch.arange(13, dtype=torch.int32, device="cuda").repeat(3, 2, 1)
    pages = torch.where(pages * 16 < n[:, None, None], pages, -1)
    a, la = svp.paged_sparse_attention(q, k, v, t, n, pages)
    b, lb = svp.paged_decode_attention(q, k, v, t, n)
    # two bf16 weights' roundings and two outputs'
    assert (a.float() - b.float()).abs().max() <= 4 * 2.0 ** -8 * 4.0
    assert (la - lb).abs().max() <= 2.0 ** -16


@pytest.mark.parametrize("dtype", DTYPES)
def test_sparse_bad_data(svp, dtype):
    """Entries past the sequence and bad ids are skipped, bad lengths leave
    their rows alone."""
    rng = np.random.default_rng(24)
    lens = np.array([40, 40, 2, 65, 0], np.int32)
    table = np.array([[0, 1, 2, 7], [9, 3, -1, 7]] + [[0, 1, 2, 3]] * 3, np.int32)
    k, v = (R.make_cache(rng, dtype, 8, 1, 64, SCALE.get(dtype, 1.0)) for _ in range(2))
    ks = SCALE.get(dtype, 1.0)
    lists = np.array([[[0, 3, 2, 1]], [[0, 1, 2, 2 ** 31 - 1]]] + [[[0, 1, 2, 3]]] * 3, np.int32)
    q = R.bf16(rng.standard_normal((5, 3, 2, 64)))
    qg = R.to_gpu(q.astype(np.float32), _io(dtype))
    import torch
    out = torch.full_like(qg, 7.0)
    lse = torch.full((5, 3, 2), 7.0, device="cuda")
    svp.paged_sparse_attention(
        qg, _gpu_cache(k, dtype), _gpu_cache(v, dtype), R.to_gpu(table), R.to_gpu(lens),
        R.to_gpu(lists), scale=0.125, out=out, lse=lse, k_scale=ks, v_scale=ks)
    assert svp.read_device_status() == 1 | 2
    assert (out[2:] == 7).all() and (lse[2:] == 7).all()
    lists[0, 0, 1], lists[1, 0] = -1, [1, -1, -1, -1]
    ref = G.sparse_attention(q[:2], R.values(k, dtype, 64, ks), R.values(v, dtype, 64, ks),
                             0.125, lens[:2], table[:2], lists[:2])
    _check(dtype, 64, out[:2], lse[:2], ref)


@pytest.mark.parametrize("dtype", DTYPES)
def test_sparse_extreme_scores(svp, dtype):
    """Scores of 1e4 and more, both signs, a scale of zero, zero rows, tiny
    rows, and NaN rows that leave the others alone."""
    rng = np.random.default_rng(25)
    for scale, gain in ((60.0, 1.0), (-60.0, 1.0), (0.0, 1.0), (0.1, 1e-30), (1e-3, 1e30)):
        q = rng.standard_normal((3, 2, 4, 64)) * gain
        q[1, 0] = 0.0
        out, lse, ref = _sparse(svp, rng, dtype, 64, 2, 2, 2, [64, 100, 130], 5,
                                scale=scale, q=q)
        _check(dtype, 64, out, lse, ref)
    q = rng.standard_normal((3, 2, 4, 64))
    q[0, 1, 2] = np.nan
    q[2, 0, 1, 5] = np.nan
    out, lse, ref = _sparse(svp, rng, dtype, 64, 2, 2, 2, [64, 100, 130], 5, 1, q=q)
    bad = np.isnan(q).any(-1)
    assert np.isnan(_f64(out)[bad]).all() and np.isnan(lse.cpu().numpy()[bad]).all()
    clean = [np.where(bad[..., None] if r.ndim == 4 else bad, 0.0, r) for r in ref]
    out = out.masked_fill(R.to_gpu(bad)[..., None], 0.0)
    lse = lse.masked_fill(R.to_gpu(bad), 0.0)
    _check(dtype, 64, out, lse, clean)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sparse_infinite_keys(svp, dtype):
    """A key of -inf products has no weight; one of +inf makes NaN."""
    import torch
    k = torch.zeros((2, 1, 16, 64), device="cuda")
    v = torch.randn((2, 1, 16, 64), device="cuda")
    k[0, 0, 3, 0] = -float("inf")
    k, v = (x.to(torch.bfloat16 if dtype == "bf16" else torch.float32) for x in (k, v))
    q = torch.zeros((1, 1, 1, 64), device="cuda", dtype=k.dtype)
    q[..., 0] = 1.0
    t = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    n = torch.tensor([32], dtype=torch.int32, device="cuda")
    pages = torch.tensor([[[0, 1]]], dtype=torch.int32, device="cuda")
    out, lse = svp.paged_sparse_attention(q, k, v, t, n, pages)
    keep = torch.arange(32, device="cuda") != 3
    want = v[:, 0].flatten(0, 1).float()[keep].mean(0)
    assert (out[0, 0, 0].float() - want).abs().max() <= 2.0 ** -7 * 4
    assert abs(float(lse) - np.log(31)) < 1e-5
    out, lse = svp.paged_sparse_attention(-q, k, v, t, n, pages)
    assert torch.isnan(out).all()


def test_sparse_offsets_beyond_4_gb(svp):
    """Pages whose bytes start past 2^32 and 2^33."""
    import torch
    nb, hkv, d = 300_000, 8, 128   # 9.8 GB a side
    k = torch.empty((nb, hkv, 16, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    ids = torch.tensor([299_999, 7, 140_000, 262_144], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [torch.randn((4, hkv, 16, d), device="cuda", generator=g).bfloat16()
            for _ in range(2)]
    k[ids], v[ids] = rows
    q = torch.randn((1, 1, hkv, d), device="cuda", generator=g).bfloat16()
    t, n = ids.int()[None], torch.tensor([60], dtype=torch.int32, device="cuda")
    pages = torch.arange(4, dtype=torch.int32, device="cuda").repeat(1, hkv, 1)
    bnd = torch.empty((nb, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    out, lse = svp.paged_sparse_attention(q, k, v, t, n, pages)
    svp.kv_page_bounds(k, t, n, bnd)
    s = svp.paged_page_scores(q, bnd, t, n)
    small = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    b2 = torch.empty((4, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    o2, l2 = svp.paged_sparse_attention(q, *rows, small, n, pages)
    svp.kv_page_bounds(rows[0], small, n, b2)
    assert svp.read_device_status() == 0
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert torch.equal(bnd[ids], b2)
    assert torch.equal(s, svp.paged_page_scores(q, b2, small, n))


def test_captured_and_on_another_stream(svp):
    """The four calls captured as a graph and replayed over other data, beside
    a second graph of the same calls on another stream."""
    import torch
    rng = np.random.default_rng(31)
    lens = np.array([500, 300, 40], np.int32)
    table, total, _ = R.pages(rng, lens)

    def program():
        g = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 30)))
        k, v = (torch.randn((total, 2, 16, 128), device="cuda", generator=g).bfloat16()
                for _ in range(2))
        q = torch.randn((3, 2, 8, 128), device="cuda", generator=g).bfloat16()
        b = torch.zeros((total, 2, 2, 128), dtype=torch.bfloat16, device="cuda")
        t, n = R.to_gpu(table), R.to_gpu(lens)

        def step():
            svp.kv_page_bounds(k, t, n, b)
            s = svp.paged_page_scores(q, b, t, n)
            p = svp.paged_select_pages(s, n, 6, 1, 2)
            return (p,) + svp.paged_sparse_attention(q, k, v, t, n, p)
        return step, (k, v, q)

    made = []
    for _ in range(2):
        step, data = program()
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        stream = torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            held = step()
        made.append((graph, stream, step, data, held))
    for turn in range(3):
        for graph, stream, step, data, held in made:
            for x in data:
                x.copy_(torch.randn_like(x.float()) * (turn + 1))
        torch.cuda.synchronize()
        for graph, stream, *_ in made:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for graph, stream, step, data, held in made:
            got = [x.clone() for x in held]
            for x, y in zip(got, step()):
                assert torch.equal(x, y)
    assert svp.read_device_status() == 0


def test_own_outputs_and_streams(svp):
    """Outputs the caller made, a stream given by name, and its refusals."""
    import torch
    k = torch.randn((4, 2, 16, 64), device="cuda")
    q = torch.randn((1, 1, 2, 64), device="cuda")
    t = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    n = torch.tensor([64], dtype=torch.int32, device="cuda")
    b = torch.zeros((4, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.empty((1, 2, 4), device="cuda")
    p = torch.empty((1, 2, 3), dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((1, 1, 2), device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    svp.kv_page_bounds(k, t, n, b, stream=stream)
    assert svp.paged_page_scores(q, b, t, n, scores=s, stream=stream).data_ptr() == s.data_ptr()
    assert svp.paged_select_pages(s, n, 3, 1, 1, pages=p, stream=stream).data_ptr() == p.data_ptr()
    r = svp.paged_sparse_attention(q, k, k, t, n, p, out=out, lse=lse, stream=stream)
    assert r[0].data_ptr() == out.data_ptr() and r[1].data_ptr() == lse.data_ptr()
    stream.synchronize()
    ref = G.sparse_attention(*(x.double().cpu().numpy() for x in (q, k, k)), 0.125,
                             [64], t.cpu().numpy(), p.cpu().numpy())
    _check("f32", 64, out, lse, ref)
    for bad in (dict(k_cache=k.transpose(0, 1)), dict(pages=p.long()), dict(pages=p[..., 0]),
                dict(q=q[..., :32]), dict(q=q.bfloat16()), dict(seq_lens=n.repeat(2)),
                dict(out=out.bfloat16()), dict(pages=p[:, :1]), dict(v_cache=k[:2])):
        args = dict(q=q, k_cache=k, v_cache=k, block_table=t, seq_lens=n, pages=p)
        args.update(bad)
        with pytest.raises(ValueError):
            svp.paged_sparse_attention(**args)
    with pytest.raises(svp.SvpError):
        svp.paged_select_pages(s, n, 3, 2, 2)
    with pytest.raises(svp.SvpError):
        svp.paged_sparse_attention(q, k, k, t, n, p[..., :0].contiguous())
    for bad in (b.float(), b[:, :1], b[:, :, :1].contiguous()):
        with pytest.raises((ValueError, svp.SvpError)):
            svp.paged_page_scores(q, bad, t, n)
    # nothing to do
    e = svp.paged_sparse_attention(q[:0], k, k, t[:0], n[:0], p[:0])
    assert e[0].shape == (0, 1, 2, 64) and svp.paged_page_scores(
        q[:0], b, t[:0], n[:0]).shape == (0, 2, 4)


def test_repeats_are_bitwise_equal(svp):
    import torch
    rng = np.random.default_rng(41)
    lens = np.array([2000, 1500], np.int32)
    table, total, _ = R.pages(rng, lens)
    k, v = (R.to_gpu(R.make_cache(rng, "bf16", total, 4, 128), "bf16") for _ in range(2))
    q = R.to_gpu(rng.standard_normal((2, 5, 16, 128)).astype(np.float32), "bf16")
    t, n = R.to_gpu(table), R.to_gpu(lens)
    pages = R.to_gpu(_lists(rng, lens, 4, 80))
    first = svp.paged_sparse_attention(q, k, v, t, n, pages)
    for _ in range(5):
        for a, b in zip(first, svp.paged_sparse_attention(q, k, v, t, n, pages)):
            assert torch.equal(a, b)
