"""The 4-bit cache on the GPU: the quantising append and the gather byte for
byte, and attention over the cache against the 64-bit definition.

Tolerances of attention, from the arithmetic (u = 2^-24, an fp32 half step):
code * scale is exact in fp16 and Q is exact in fp16 but for values 2^-28 of
the row's largest, so a score is off by the fp32 summation of D products,
at most delta = 2 D u sum|q||k| |scale| (matrix instructions may truncate:
one whole step per addition), and by the scaled value's own roundings,
8 u |score|.  Weights are then off by a factor 1 + 2 delta, fp16 weights by
2^-11 more, each key's V counts with its weight: out is off by at most
(2 delta + 2^-11 + 2^-16) max|v| + 2^-8 |out| (bf16 output), the lse by
2 delta + 2^-18 (exp2 and log2 approximations) + 4 u |lse|."""
import ctypes

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


def _check(out, lse, ref, d):
    o_ref, l_ref, mag, vmax = ref
    u = 2.0 ** -24
    delta = 2 * d * u * mag + 8 * u * (mag + np.abs(l_ref))
    tol_o = ((2 * delta + 2.0 ** -11 + 2.0 ** -16) * vmax)[..., None] + 2.0 ** -8 * np.abs(o_ref)
    tol_l = 2 * delta + 2.0 ** -18 + 4 * u * np.abs(l_ref)
    eo = np.abs(out.double().cpu().numpy() - o_ref)
    el = np.abs(lse.double().cpu().numpy() - l_ref)
    assert (eo <= tol_o).all(), (eo / tol_o).max()
    assert (el <= tol_l).all(), (el / tol_l).max()


def _inputs(seed, lens, hq, hkv, d, q_len, ks=1.0, vs=1.0, width=None):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    table, total, _ = R.pages(rng, lens, spare=2, width=width)
    kc = R.make_cache(rng, "fp4", total, hkv, d, ks, lens, table)
    vc = R.make_cache(rng, "fp4", total, hkv, d, vs, lens, table)
    q = R.bf16(rng.standard_normal((len(lens), q_len, hq, d)))
    return q, kc, vc, table, lens


def _dims(bd, batch, hq, cache, max_blocks, split_pages=0, kernel_path=0):
    nb, hkv, page, row = cache.shape
    return bd.SvpDims(batch, hq, hkv, row * 16 // 9, page, max_blocks, nb,
                      bd.SVP_FP4_E2M1, None, 0, split_pages, kernel_path, 1.0, 1.0)


def _reference(q, kc, vc, d, scale, lens, table, ks, vs, **mask):
    with np.errstate(invalid="ignore"):
        return R.attention(q, R.values(kc, "fp4", d, ks), R.values(vc, "fp4", d, vs),
                           scale, lens, table, **mask)


# ------------------------------------------------------------- the append

@pytest.mark.parametrize("d,hkv,n_new,lens,ks", [
    (128, 3, 1, [1, 16, 17, 40], 1.0),
    (64, 2, 5, [5, 33, 64], 0.0371),
    (128, 8, 64, [64, 200], 0.4),
    (64, 1, 17, [17], 2.0 ** -7),
])
def test_append_and_gather(svp, d, hkv, n_new, lens, ks):
    import torch
    rng = np.random.default_rng(d + n_new)
    lens = np.asarray(lens, np.int32)
    table, total, _ = R.pages(rng, lens)
    vs = 1.3 * ks
    kc = rng.integers(0, 256, (total, hkv, 16, 9 * d // 16)).astype(np.uint8)
    vc = rng.integers(0, 256, kc.shape).astype(np.uint8)
    new = [R.bf16(rng.standard_normal((len(lens), n_new, hkv, d)) *
                  np.exp(3 * rng.standard_normal((len(lens), n_new, hkv, 1))))
           for _ in range(2)]
    gk, gv = R.to_gpu(kc), R.to_gpu(vc)
    gt, gl = R.to_gpu(table), R.to_gpu(lens)
    svp.kv_append(R.to_gpu(new[0], "bf16"), R.to_gpu(new[1], "bf16"), gk, gv, gt,
                  gl, k_scale=ks, v_scale=vs)
    for cache, x, s in ((kc, new[0], ks), (vc, new[1], vs)):
        rows = R.quantise(x, s)
        for b, L in enumerate(lens):
            for i in range(n_new):
                j = L - n_new + i
                cache[table[b, j // 16], :, j % 16] = rows[b, i]
    assert np.array_equal(gk.cpu().numpy(), kc)     # other rows untouched
    assert np.array_equal(gv.cpu().numpy(), vc)
    got_k, got_v = svp.kv_gather(gk, gv, gt, gl, n_new, k_scale=ks, v_scale=vs)
    for got, x, s in ((got_k, new[0], ks), (got_v, new[1], vs)):
        # fp32 of code * scale * factor, then bf16: two roundings
        ref = R.values(R.quantise(x, s), "fp4", d, float(np.float32(s)))
        err = np.abs(got.double().cpu().numpy() - ref)
        assert (err <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref)).all()
    assert svp.read_device_status() == 0


def test_append_extremes(svp):
    """Zero blocks, values below the smallest scale, saturation, ties, signs
    of zero, infinities and NaN."""
    import torch
    d = 64
    x = np.zeros((1, 1, 4, d))
    x[0, 0, 0, 16:32] = R.bf16(np.linspace(-1, 1, 16) * 2.0 ** -14)
    x[0, 0, 0, 32:48] = R.bf16(np.linspace(-3e38, 3e38, 16))
    x[0, 0, 0, 48:64] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75,
                         -1.25, -1.75, -2.5, -3.5, -5, -6]   # ties, scale 1
    x[0, 0, 1] = R.bf16(np.arange(-32, 32) * 2.0 ** -9)
    x[0, 0, 2, :16] = 2.0 ** -133                             # bf16 subnormal
    x[0, 0, 3] = -2688.0
    t = R.to_gpu(x, "bf16")
    t[0, 0, 2, 20] = float("inf")
    t[0, 0, 2, 21] = float("-inf")
    t[0, 0, 2, 40] = float("nan")
    t[0, 0, 2, 41] = 1.5
    gk = torch.zeros((1, 4, 16, svp.fp4_row_bytes(d)), dtype=torch.uint8, device="cuda")
    gv = torch.zeros_like(gk)
    gt = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    gl = torch.ones(1, dtype=torch.int32, device="cuda")
    svp.kv_append(t, t, gk, gv, gt, gl)
    got = gk[0, :, 0].cpu().numpy()
    ref = R.quantise(x[0, 0], 1.0)
    for h in (0, 1, 3):
        assert np.array_equal(got[h], ref[h]), h
    assert np.array_equal(gv.cpu().numpy(), gk.cpu().numpy())
    v = R.values(got, "fp4", d)
    assert (v[2, :16] == 0).all()
    assert v[2, 20] == 6 * 448 and v[2, 21] == -6 * 448
    assert v[2, 40] == 6 * 0.25 and v[2, 41] == 1.5           # NaN: largest code


@pytest.mark.parametrize("ks", [1.0, 0.5, 3.0, 0.1, 1e-3, 7.0, 1e-30, 3e37])
def test_append_near_every_rounding_border(svp, ks):
    """Byte for byte where a quotient lies on, or one bf16 step beside, a
    border between codes or between block scales; and every bf16 mantissa as
    a block's largest value."""
    import torch
    d, hkv = 128, 4
    rng = np.random.default_rng(6)
    f32 = np.float32
    blocks = []
    mant = (1 + np.arange(128) / 128.0)
    tops = np.concatenate([mant * 2.0 ** e for e in (-12, -9, -3, 0, 4, 11, 12)])
    # largest values whose sixth is a border between two E4M3 scales
    mids = (R.E4M3[:126] + R.E4M3[1:127]) / 2 * 6
    tops = np.concatenate([tops, mids])
    for top in tops:
        top = min(float(top) * float(f32(ks)), 3e38)
        top = float(R.bf16(np.array([top]))[0])
        y = float(f32(f32(top) / f32(ks)))
        sc = R.E4M3[max(int(R.e4m3_code(np.array([float(f32(y) / f32(6))]))[0]), 1)]
        near = []
        for lo, hi in zip(R.E2M1[:-1], R.E2M1[1:]):
            x = float(R.bf16(np.array([min((lo + hi) / 2 * sc * ks, 3e38)]))[0])
            near += [x, np.nextafter(f32(x), f32(0)) if x else 0.0]
        x = np.array([top] + near + [0.0] * 16)[:16]
        x = np.minimum(np.abs(R.bf16(x)), top)
        # a bf16 step up or down, and signs
        u = x.astype(f32).view(np.uint32) + (rng.integers(-1, 2, 16) * 65536).astype(np.int64)
        x = np.maximum(u, 0).astype(np.uint32).view(f32).astype(np.float64)
        x = np.minimum(x, top)
        x[0] = top
        blocks.append(rng.permutation(x) * rng.choice([-1.0, 1.0], 16))
    per = hkv * d // 16
    n = -(-len(blocks) // per)
    blocks += [np.zeros(16)] * (n * per - len(blocks))
    x = R.bf16(np.stack(blocks).reshape(1, n, hkv, d))
    t = R.to_gpu(x, "bf16")
    width = -(-n // 16)
    gk = torch.zeros((width, hkv, 16, svp.fp4_row_bytes(d)), dtype=torch.uint8, device="cuda")
    gv = torch.zeros_like(gk)
    gt = torch.arange(width, dtype=torch.int32, device="cuda").view(1, -1)
    gl = torch.full((1,), n, dtype=torch.int32, device="cuda")
    svp.kv_append(t, t, gk, gv, gt, gl, k_scale=ks, v_scale=ks)
    got = gk.cpu().numpy().transpose(0, 2, 1, 3).reshape(width * 16, hkv, -1)[:n]
    with np.errstate(over="ignore"):
        want = R.quantise(x[0], ks)
    # (a zero quotient keeps its sign here, not in the reference)
    zero = np.zeros(x[0].shape, np.uint8)
    zero[(x[0].astype(f32) / f32(ks) == 0) & np.signbit(x[0])] = 8
    want[..., :d // 2] |= zero[..., 0::2] | (zero[..., 1::2] << 4)
    assert np.array_equal(got, want)
    assert torch.equal(gk, gv)


def test_append_of_random_bit_patterns(svp):
    """Finite bf16 patterns at random, against factors at random."""
    import torch
    rng = np.random.default_rng(9)
    B, n, hkv, d = 8, 64, 2, 64
    gt = torch.arange(B * n // 16, dtype=torch.int32, device="cuda").view(B, -1)
    gl = torch.full((B,), n, dtype=torch.int32, device="cuda")
    for ks in np.exp(rng.uniform(-80, 80, 6)).astype(np.float32):
        u = rng.integers(0, 65536, (B, n, hkv, d)).astype(np.uint32) << 16
        with np.errstate(invalid="ignore"):
            x = u.view(np.float32).astype(np.float64)
        x = np.where(np.isfinite(x), x, 1.0)
        # half of the rows within a factor of 64, where the codes vary
        y = float(ks) * R.bf16(rng.standard_normal(x.shape) * np.exp(rng.uniform(-4, 4, x.shape)))
        x = np.where(rng.random((B, n, hkv, 1)) < 0.5, R.bf16(np.clip(y, -3e38, 3e38)), x)
        t = R.to_gpu(x, "bf16")
        gk = torch.zeros((B * n // 16, hkv, 16, svp.fp4_row_bytes(d)), dtype=torch.uint8,
                         device="cuda")
        gv = torch.zeros_like(gk)
        svp.kv_append(t, t, gk, gv, gt, gl, k_scale=float(ks), v_scale=float(ks))
        got = gk.cpu().numpy().transpose(0, 2, 1, 3).reshape(B, n, hkv, -1)
        with np.errstate(over="ignore"):
            want = R.quantise(x, ks)
        # (values: a zero's sign does not count)
        assert np.array_equal(got[..., d // 2:], want[..., d // 2:])
        assert np.array_equal(R.values(got, "fp4", d), R.values(want, "fp4", d))


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128), ("fp8", 64),
                                     ("fp8", 128), ("fp4", 64), ("fp4", 128)])
def test_gather_positions(svp, dtype, d):
    """starts before, inside and past the sequence, an empty sequence."""
    import torch
    rng = np.random.default_rng(4)
    lens = np.array([0, 1, 16, 50, 33], np.int32)
    starts = np.array([0, -3, 15, 40, 33], np.int32)
    table, total, _ = R.pages(rng, lens)
    scale = 0.07 if dtype in ("fp4", "fp8") else 1.0
    kc = R.make_cache(rng, dtype, total, 3, d, scale, lens, table)
    vc = R.make_cache(rng, dtype, total, 3, d, scale, lens, table)
    io = "bf16" if dtype == "bf16" else None
    n = 21
    k, v = svp.kv_gather(R.to_gpu(kc, io), R.to_gpu(vc, io), R.to_gpu(table),
                         R.to_gpu(lens), n, starts=R.to_gpu(starts),
                         k_scale=scale, v_scale=scale)
    assert k.dtype == (torch.float32 if dtype == "f32" else torch.bfloat16)
    for got, cache in ((k, kc), (v, vc)):
        with np.errstate(invalid="ignore"):
            val = R.values(cache, dtype, d, float(np.float32(scale)))
        ref = np.zeros((len(lens), n, 3, d))
        for b in range(len(lens)):
            for i in range(n):
                j = starts[b] + i
                if 0 <= j < lens[b]:
                    ref[b, i] = val[table[b, j // 16], :, j % 16]
        err = np.abs(got.double().cpu().numpy() - ref)
        exact = dtype in ("f32", "bf16")
        assert (err <= (0 if exact else 2.0 ** -8 + 2.0 ** -23) * np.abs(ref)).all()
    assert svp.read_device_status() == 0


# -------------------------------------------------------------- attention

CASES = [
    # d, hq, hkv, q_len, lens, mask, split_pages, k_scale
    (128, 4, 4, 1, [1, 2, 15, 16, 17, 31, 32, 33, 300], {}, 0, 1.0),
    (64, 4, 2, 1, [1, 5, 16, 47, 129, 260], {}, 1, 0.0371),
    (128, 8, 1, 1, [700, 9], {}, 2, 1.0),                       # 8 rows
    (128, 16, 4, 3, [3, 4, 19, 500], {}, 0, 0.4),               # 12 rows
    (128, 32, 8, 5, [5, 64, 333], {}, 1, 1.0),                  # 20 rows
    (64, 14, 2, 4, [4, 18, 150], {}, 0, 1.0),                   # 28 rows
    (128, 6, 2, 16, [16, 17, 100, 290], {}, 0, 1.0),            # 48 rows
    (128, 32, 8, 15, [15, 90, 210], {}, 0, 1.0),                # 60 rows
    (64, 16, 2, 16, [16, 130], {}, 2, 1.0),                     # 128 rows
    (128, 40, 2, 5, [77], {}, 0, 1.0),                          # 100 rows
    (128, 4, 4, 1, [1, 40, 300, 301], dict(n_sink=4, window=37), 0, 1.0),
    (64, 8, 2, 4, [4, 63, 200], dict(n_sink=0, window=1), 1, 1.0),
    (128, 8, 2, 6, [6, 63, 200], dict(n_sink=17, window=33), 0, 1.0),
    (128, 32, 8, 15, [15, 16, 31, 220], "tree", 0, 1.0),
    (64, 4, 2, 7, [7, 23, 90], "tree", 1, 0.0371),
]


PATHS = {0: "auto", 2: "mma", 3: "tcgen05"}


@pytest.mark.parametrize("path", PATHS, ids=PATHS.values())
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention(svp, case, path):
    import torch
    d, hq, hkv, ql, lens, mask, split, ks = case
    if path == 3 and d != 128:
        pytest.skip("head_dim 128 only")
    vs = 0.75 * ks
    q, kc, vc, table, lens = _inputs(d + hq + ql, lens, hq, hkv, d, ql, ks, vs)
    scale = 1.0 / np.sqrt(d)
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table),
         R.to_gpu(lens)]
    fks, fvs = float(np.float32(ks)), float(np.float32(vs))
    if mask == "tree":
        tree = np.tile(R.binary_tree(ql), (len(lens), 1))
        out, lse = svp.paged_tree_attention(*g, R.to_gpu(tree), scale=scale,
                                            split_pages=split, kernel_path=path,
                                            k_scale=ks, v_scale=vs)
        mask = dict(tree=tree)
    else:
        out, lse = svp.paged_decode_attention(*g, scale=scale, split_pages=split,
                                              kernel_path=path, k_scale=ks,
                                              v_scale=vs, **mask)
    assert svp.read_device_status() == 0
    ref = _reference(q, kc, vc, d, float(np.float32(scale)), lens, table, fks, fvs, **mask)
    _check(out, lse, ref, d)


@pytest.mark.parametrize("path", [2, 3])
@pytest.mark.parametrize("gain,scale", [(1e-30, 1e28), (200.0, 1.0), (1.0, 0.0),
                                        (1.0, -0.3), (3e4, 1e-3)])
def test_query_ranges_and_scales(svp, gain, scale, path):
    """Query rows far outside fp16's range, sharp softmaxes, a zero and a
    negative scale."""
    d = 128
    q, kc, vc, table, lens = _inputs(9, [40, 150], 4, 2, d, 2)
    q = R.bf16(q * gain)
    out, lse = svp.paged_decode_attention(
        R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table),
        R.to_gpu(lens), scale=scale, kernel_path=path)
    ref = _reference(q, kc, vc, d, float(np.float32(scale)), lens, table, 1.0, 1.0)
    _check(out, lse, ref, d)


@pytest.mark.parametrize("path", [2, 3])
def test_rising_scores(svp, path):
    """Scores that grow by more than the softmax's slack from page to page:
    the reference moves at every page."""
    d = 128
    q, kc, vc, table, lens = _inputs(5, [300], 1, 1, d, 1)
    q[:] = 1.0
    ramp = np.repeat(np.linspace(-40, 40, 300)[:, None], d, 1)[:, None, :] / d
    rows = R.quantise(R.bf16(ramp), 1.0)
    for j in range(300):
        kc[table[0, j // 16], :, j % 16] = rows[j]
    out, lse = svp.paged_decode_attention(
        R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table),
        R.to_gpu(lens), scale=1.0, kernel_path=path)
    _check(out, lse, _reference(q, kc, vc, d, 1.0, lens, table, 1.0, 1.0), d)


@pytest.mark.parametrize("ql", [1, 5])
def test_many_splits_and_wide_table(svp, ql):
    """One long sequence over the whole grid (partials merged across many
    CTAs), a block table wider than any sequence, repeatable results."""
    import torch
    d = 128
    q, kc, vc, table, lens = _inputs(11, [6000, 40], 8, 2, d, ql, width=900)
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table), R.to_gpu(lens)]
    out, lse = svp.paged_decode_attention(*g, scale=0.1)
    again, lse2 = svp.paged_decode_attention(*g, scale=0.1)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    _check(out, lse, _reference(q, kc, vc, d, float(np.float32(0.1)), lens, table, 1.0, 1.0), d)


@pytest.mark.parametrize("width", [4, 40])
def test_more_sequences_than_a_launch_takes(svp, width):
    """1100 sequences, in several launches; 4 pages a sequence at most (a
    warp takes one whole) and a wide table (slices)."""
    rng = np.random.default_rng(width)
    lens = rng.integers(1, 65, 1100)
    q, kc, vc, table, lens = _inputs(5, lens, 2, 1, 64, 1, width=width)
    out, lse = svp.paged_decode_attention(
        R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table),
        R.to_gpu(lens), scale=0.125)
    assert svp.read_device_status() == 0
    _check(out, lse, _reference(q, kc, vc, 64, 0.125, lens, table, 1.0, 1.0), 64)


@pytest.mark.parametrize("d,batch,hkv,width,mask", [
    (128, 600, 1, 50, {}),       # in slices, and a launch for the 88 left
    (64, 600, 2, 31, {}),        # whole groups
    (128, 512, 12, 50, dict(n_sink=5, window=40)),
    (128, 520, 1, 50, "tree"),
], ids=["slices", "whole", "window", "tree"])
def test_wide_units(svp, d, batch, hkv, width, mask):
    """24 query rows and enough pages for the widest unit."""
    import torch
    rng = np.random.default_rng(width)
    ql, hq = 6, 4 * hkv
    lens = rng.integers(ql, 90, batch)
    lens[:3] = (ql, 31 * 16, 200)
    q, kc, vc, table, lens = _inputs(7, lens, hq, hkv, d, ql, 0.4, 0.3, width=width)
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table), R.to_gpu(lens)]
    kw = dict(scale=0.125, k_scale=0.4, v_scale=0.3)
    if mask == "tree":
        mask = dict(tree=np.tile(R.binary_tree(ql), (batch, 1)))
        call = lambda: svp.paged_tree_attention(*g, R.to_gpu(mask["tree"]), **kw)
    else:
        call = lambda: svp.paged_decode_attention(*g, **kw, **mask)
    out, lse = call()
    assert svp.read_device_status() == 0
    ref = _reference(q, kc, vc, d, 0.125, lens, table, float(np.float32(0.4)),
                     float(np.float32(0.3)), **mask)
    _check(out, lse, ref, d)
    again, _ = call()
    assert torch.equal(out, again)


@pytest.mark.parametrize("d,batch,hq,hkv,ql,width,mask", [
    (64, 1, 4, 4, 1, 16, {}),
    (128, 1, 8, 1, 1, 3, {}),
    (128, 3, 16, 2, 2, 64, {}),                # 63 pages over eight warps
    (128, 40, 16, 8, 1, 31, {}),               # four warps a group
    (128, 90, 8, 8, 1, 20, {}),                # two
    (64, 200, 8, 8, 1, 12, {}),                # one, and CTAs of twelve groups
    (128, 30, 16, 4, 5, 30, {}),
    (128, 8, 24, 4, 4, 40, dict(n_sink=3, window=100)),
    (128, 5, 16, 4, 4, 8, "tree"),
], ids=lambda x: None)
def test_whole_groups(svp, d, batch, hq, hkv, ql, width, mask):
    """Short sequences, the warps of a team with full, single and no pages;
    one sequence's length is out of range and another's page is bad."""
    import torch
    rng = np.random.default_rng(width * batch)
    lens = rng.integers(ql, 16 * width, batch)
    lens[0] = 16 * width - 5
    if batch > 2:
        lens[1:3] = (ql, min(17, 16 * width))
    q, kc, vc, table, lens = _inputs(8, lens, hq, hkv, d, ql, width=width)
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table), R.to_gpu(lens)]
    if mask == "tree":
        mask = dict(tree=np.tile(R.binary_tree(ql), (batch, 1)))
        call = lambda *a: svp.paged_tree_attention(*a, R.to_gpu(mask["tree"]), scale=0.1)
    else:
        call = lambda *a: svp.paged_decode_attention(*a, scale=0.1, **mask)
    out, lse = call(*g)
    assert svp.read_device_status() == 0 and svp.last_launch_count() == 1
    ref = _reference(q, kc, vc, d, float(np.float32(0.1)), lens, table, 1.0, 1.0, **mask)
    _check(out, lse, ref, d)
    if batch > 4:
        bad_lens, bad = lens.copy(), table.copy()
        bad_lens[3], bad[0, 0] = 10 ** 6, -7
        o2, l2 = call(*g[:3], R.to_gpu(bad), R.to_gpu(bad_lens))
        assert svp.read_device_status() == 3
        rest = [b for b in range(batch) if b not in (0, 3)]
        assert torch.equal(o2[rest], out[rest]) and torch.equal(l2[rest], lse[rest])
        assert torch.isfinite(o2[0].float()).all()


def test_stalled_whole_groups_time_out(svp):
    """The same test build over short sequences, four warps to a group: those
    with more than the two stages that arrive give up, the team meets and
    leaves the output alone; a short sequence's team is right."""
    import torch
    from spec_verify_paged_gb300 import binding as bd, build
    from test_bounded_wait import STALL_DEFINES
    stall = bd.load_library(build.build_variant("stalltest", STALL_DEFINES))
    d, batch = 128, 20
    lens = [1000] * (batch - 1) + [100]
    q, kc, vc, table, lens = _inputs(42, lens, 8, 8, d, 1)
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table), R.to_gpu(lens)]
    out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], 3.0, device="cuda")
    dims = _dims(bd, batch, 8, g[1], table.shape[1])
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert stall.paged_decode_attention(
        ctypes.byref(dims), *(t.data_ptr() for t in g), 1, 0, 0, float(np.float32(0.1)),
        out.data_ptr(), lse.data_ptr(), stream) == 0
    assert stall.svp_last_launch_count() == 1
    torch.cuda.synchronize()
    f = ctypes.c_int(0)
    assert stall.svp_read_device_status(stream, ctypes.byref(f)) == 0
    assert f.value & 8
    assert (out[:-1] == 3).all() and (lse[:-1] == 3).all()
    ref = svp.paged_decode_attention(*g, scale=0.1)
    assert torch.equal(out[-1], ref[0][-1]) and torch.equal(lse[-1], ref[1][-1])
    assert svp.read_device_status() == 0


@pytest.mark.parametrize("path", [2, 3])
def test_rows_that_see_nothing(svp, path):
    """A tree mask without any bit over a sequence of the new rows only: zero
    output and lse -inf; the other sequence is as without them."""
    import torch
    d, ql = 128, 5
    q, kc, vc, table, lens = _inputs(13, [ql, 77], 8, 2, d, ql)
    tree = np.stack([np.zeros(ql, np.int32), R.binary_tree(ql)])
    tree[0, 3] = 0b1000                       # one row of it sees itself
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table), R.to_gpu(lens)]
    mask = R.to_gpu(tree)
    out, lse = svp.paged_tree_attention(*g, mask, scale=0.1, kernel_path=path)
    none = [0, 1, 2, 4]
    assert (out[0, none] == 0).all() and (lse[0, none] == -float("inf")).all()
    s = float(np.float32(0.1))
    k3 = R.values(kc, "fp4", d)[table[0, 0], :, 3]
    v3 = R.values(vc, "fp4", d)[table[0, 0], :, 3]
    for h in range(8):
        x = float(k3[h // 4] @ q[0, 3, h]) * s
        assert abs(float(lse[0, 3, h]) - x) <= 2.0 ** -16 * (1 + np.abs(k3[h // 4]) @ np.abs(q[0, 3, h]))
        got = out[0, 3, h].double().cpu().numpy()
        assert (np.abs(got - v3[h // 4]) <= (2.0 ** -8 + 2.0 ** -9) * np.abs(v3[h // 4])).all()
    ref = _reference(q[1:], kc, vc, d, s, lens[1:], table[1:], 1.0, 1.0, tree=tree[1:])
    _check(out[1:], lse[1:], ref, d)
    # the score update of the same rows: rows that see nothing add nothing
    scores = torch.zeros((kc.shape[0], 2, 16), device="cuda")
    svp.paged_score_update(g[0], g[1], lse, g[3], g[4], scores, scale=0.1, tree_mask=mask)
    first = scores[int(table[0, 0])].cpu().numpy()
    assert (first[:, [0, 1, 2] + list(range(4, 16))] == 0).all()
    # four rows of weight exp(0): the score and the lse each round
    assert np.abs(first[:, 3] - 4).max() < 1e-3
    if hasattr(torch, "uint32"):
        o2, l2 = svp.paged_tree_attention(*g, mask.view(torch.uint32), scale=0.1,
                                          kernel_path=path)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_offsets_beyond_32_bits(svp):
    """Pages on both sides of 4 GB of cache: append, attention, gather, score
    update and eviction give what they give on a small cache."""
    import torch
    d, hkv, hq = 128, 8, 16
    total = 5 * 10 ** 9 // (hkv * 16 * 72)
    free, _ = torch.cuda.mem_get_info()
    if free < 14 * 10 ** 9:
        pytest.skip("not enough device memory")
    rng = np.random.default_rng(12)
    lens = np.array([200, 64], np.int32)
    small = rng.permutation(26).astype(np.int32).reshape(2, 13)
    far = np.sort(rng.choice(np.r_[0:40, total - 60:total], 26, replace=False))
    far = rng.permutation(far).astype(np.int32)
    x = [torch.randn((2, 64, hkv, d), device="cuda").to(torch.bfloat16) for _ in range(2)]
    q = torch.randn((2, 1, hq, d), device="cuda").to(torch.bfloat16)
    results = []
    for n, ids in ((26, np.arange(26)), (total, far)):
        kc = torch.zeros((n, hkv, 16, 72), dtype=torch.uint8, device="cuda")
        vc = torch.zeros_like(kc)
        s = torch.zeros((n, hkv, 16), device="cuda")
        gt = R.to_gpu(ids[small].astype(np.int32))
        for L in (64, 128, 192, 200):          # sequence 0 grows
            svp.kv_append(*x, kc, vc, gt, R.to_gpu(np.array([L, 64], np.int32)))
        gl = R.to_gpu(lens)
        out, lse = svp.paged_decode_attention(q, kc, vc, gt, gl)
        svp.paged_score_update(q, kc, lse, gt, gl, s)
        rows = svp.kv_gather(kc, vc, gt, gl, 200)
        kept, new = svp.kv_evict(kc, vc, s, gt, gl, 48, 4, 8)
        after = svp.kv_gather(kc, vc, gt, new, 48)
        at = R.to_gpu(ids.astype(np.int64))
        results.append([out, lse, *rows, kept, new, *after, s[at], kc[at], vc[at]])
        assert svp.read_device_status() == 0
        del kc, vc, s
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_calls_on_a_stream_of_their_own(svp):
    """The whole step on a side stream while the current one is busy, outputs
    made by the call: as on the current stream."""
    import torch
    d, hkv, hq = 128, 2, 8
    q, kc, vc, table, lens = _inputs(41, [300, 90], hq, hkv, d, 1)
    rng = np.random.default_rng(1)
    new = [R.to_gpu(R.bf16(rng.standard_normal((2, 1, hkv, d))), "bf16") for _ in range(2)]
    gq, gt, gl = R.to_gpu(q, "bf16"), R.to_gpu(table), R.to_gpu(lens)
    side = torch.cuda.Stream()
    results = []
    for stream in (None, side):
        k, v = R.to_gpu(kc), R.to_gpu(vc)
        s = torch.zeros((kc.shape[0], hkv, 16), device="cuda")
        torch.cuda.synchronize()
        if stream is not None:     # the current stream lags behind
            busy = torch.randn((4096, 4096), device="cuda")
            for _ in range(20):
                busy = busy @ busy * 1e-3
        svp.kv_append(*new, k, v, gt, gl, stream=stream)
        out, lse = svp.paged_decode_attention(gq, k, v, gt, gl, stream=stream)
        svp.paged_score_update(gq, k, lse, gt, gl, s, stream=stream)
        kept, n = svp.kv_evict(k, v, s, gt, gl, 80, 4, 8, stream=stream)
        rows = svp.kv_gather(k, v, gt, n, 80, stream=stream)
        torch.cuda.synchronize()
        results.append([out, lse, s, kept, n, *rows, k, v])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_empty_calls_and_layouts(svp):
    """No rows, no sequences; a transposed cache, a sliced query and a wrong
    device are refused."""
    import torch
    q, kc, vc, table, lens = _inputs(43, [30, 9], 4, 2, 64, 1)
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table), R.to_gpu(lens)]
    k, v = svp.kv_gather(*g[1:], 0)
    assert tuple(k.shape) == (2, 0, 2, 64) == tuple(v.shape)
    none = [g[0][:0], *g[1:3], g[3][:0], g[4][:0]]
    out, lse = svp.paged_decode_attention(*none)
    assert out.shape[0] == 0 and lse.shape[0] == 0
    s = torch.ones((kc.shape[0], 2, 16), device="cuda")
    svp.paged_score_update(none[0], none[1], lse, *none[3:], s)
    kept, n = svp.kv_evict(*none[1:3], s, *none[3:], 8)
    assert kept.shape[0] == 0 and n.shape[0] == 0 and (s == 1).all()
    wide = torch.zeros((2, 1, 8, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        svp.paged_decode_attention(wide[:, :, ::2], *g[1:])
    with pytest.raises(ValueError):
        svp.kv_gather(g[1].transpose(0, 1), g[2].transpose(0, 1), *g[3:], 1)
    with pytest.raises(ValueError):
        svp.kv_gather(*g[1:4], g[4].cpu(), 1)
    with pytest.raises(ValueError):
        svp.paged_decode_attention(*g[:4], g[4].long())
    with pytest.raises(ValueError):
        svp.kv_evict(*g[1:3], s.double(), *g[3:], 8)
    with pytest.raises(TypeError):
        svp.kv_gather(g[1], None, *g[3:], 1)
    assert svp.read_device_status() == 0


@pytest.mark.parametrize("path", [2, 3])
def test_bad_pages_and_lengths_are_flagged(svp, path):
    """A bad page is left out, a bad sequence is left as it was; the others
    are right."""
    import torch
    d = 128
    q, kc, vc, table, lens = _inputs(3, [64, 50, 40], 4, 4, d, 1)
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc)]
    bad = table.copy()
    bad[0, 1] = 10 ** 6
    bad_lens = lens.copy()
    bad_lens[2] = 10 ** 6
    out = torch.full((3, 1, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 1, 4), 7.0, device="cuda")
    svp.paged_decode_attention(*g, R.to_gpu(bad), R.to_gpu(bad_lens), scale=0.1,
                               out=out, lse=lse, kernel_path=path)
    assert svp.read_device_status() == 3      # bad block id, bad length
    assert (out[2] == 7).all() and (lse[2] == 7).all()
    ref = _reference(q[1:2], kc, vc, d, float(np.float32(0.1)), lens[1:2], table[1:2], 1.0, 1.0)
    _check(out[1:2], lse[1:2], ref, d)
    keep = np.r_[0:16, 32:64]                 # sequence 0 without its page 1
    short = np.stack([table[0, [0, 2, 3]]])
    ref = _reference(q[:1], kc, vc, d, float(np.float32(0.1)), np.array([len(keep)]),
                     short, 1.0, 1.0)
    _check(out[:1], lse[:1], ref, d)


def test_own_stream_and_captured_graphs(svp):
    """Calls on a stream of their own, and two captured graphs whose calls
    have workspaces of their own, replayed in either order and at once."""
    import torch
    d = 128
    sets = [_inputs(s, lens, 8, 2, d, 4) for s, lens in ((1, [600, 30]), (2, [40, 2000]))]
    gpu, graphs, outs = [], [], []
    for q, kc, vc, table, lens in sets:
        gpu.append([R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table),
                    R.to_gpu(lens)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = [svp.paged_decode_attention(*g, scale=0.1, stream=side) for g in gpu]
    side.synchronize()
    for g in gpu:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(svp.paged_decode_attention(*g, scale=0.1))
        graphs.append(gr)
    for order in ((0, 1), (1, 0)):
        for o, l in outs:
            o.fill_(9)
            l.fill_(9)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for i in order:
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for (o, l), (fo, fl) in zip(outs, first):
            assert torch.equal(o, fo) and torch.equal(l, fl)
    for (q, kc, vc, table, lens), (o, l) in zip(sets, first):
        _check(o, l, _reference(q, kc, vc, d, float(np.float32(0.1)), lens, table, 1.0, 1.0), d)
    assert svp.read_device_status() == 0


def test_noalloc_and_caller_workspace(svp):
    import torch
    from spec_verify_paged_gb300 import binding as bd
    d = 64
    q, kc, vc, table, lens = _inputs(21, [500, 17, 90], 6, 3, d, 2)
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table), R.to_gpu(lens)]
    out, lse = svp.paged_decode_attention(*g, scale=0.1)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    o2, l2 = svp.paged_decode_attention(*g, scale=0.1, workspace=ws)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    lib = svp.load_library()
    dims = _dims(bd, 3, 6, g[1], table.shape[1])
    o3, l3 = torch.zeros_like(out), torch.zeros_like(lse)
    st = lib.paged_decode_attention_noalloc(
        ctypes.byref(dims), *(t.data_ptr() for t in g), 2, 0, 0,
        float(np.float32(0.1)), o3.data_ptr(), l3.data_ptr(),
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(out, o3) and torch.equal(lse, l3)
    with pytest.raises(svp.SvpError) as e:
        svp.paged_decode_attention(*g, workspace=ws[:64])
    assert e.value.status == -4


def test_step_runner_over_a_4bit_cache(svp):
    """The graph-captured decode step appends to and reads a 4-bit cache:
    bit-identical to the plain calls."""
    import torch
    d, hq, hkv, ql, B = 128, 8, 2, 3, 2
    q, kc, vc, table, lens = _inputs(31, [70, 200], hq, hkv, d, ql)
    rng = np.random.default_rng(8)
    ks, vs = 0.4, 0.3
    runs = [[R.to_gpu(kc), R.to_gpu(vc)] for _ in range(2)]
    run = svp.StepRunner(*runs[0], B, hq, ql, table.shape[1], k_scale=ks, v_scale=vs)
    try:
        for step in range(3):
            new = [rng.standard_normal((B, ql, h, d)) for h in (hq, hkv, hkv)]
            t = [R.to_gpu(x, "bf16") for x in new]
            slot = step % 2
            for name, x in zip(("q", "k_new", "v_new"), t):
                run.host(slot, name)[:] = x.view(torch.int16).cpu().numpy().view(np.uint16)
            run.host(slot, "block_table")[:] = table
            run.host(slot, "seq_lens")[:] = lens
            run.launch(slot)
            run.wait(slot)
            gt, gl = R.to_gpu(table), R.to_gpu(lens)
            svp.kv_append(t[1], t[2], *runs[1], gt, gl, k_scale=ks, v_scale=vs)
            out, lse = svp.paged_decode_attention(t[0], *runs[1], gt, gl,
                                                  k_scale=ks, v_scale=vs)
            got = torch.from_numpy(run.host(slot, "out").view(np.int16).copy())
            assert torch.equal(got, out.view(torch.int16).cpu())
            assert np.array_equal(run.host(slot, "lse"), lse.cpu().numpy())
        for a, b in zip(*runs):
            assert torch.equal(a, b)
    finally:
        run.close()
    assert svp.read_device_status() == 0


@pytest.mark.parametrize("path", [2, 3])
def test_stalled_producer_times_out(svp, path):
    """A test build whose producers stop: every role's bounded wait runs out,
    the call returns with the flag set, and the next call is right."""
    import torch
    from spec_verify_paged_gb300 import binding as bd, build
    from test_bounded_wait import STALL_DEFINES
    stall = bd.load_library(build.build_variant("stalltest", STALL_DEFINES))
    d = 128
    q, kc, vc, table, lens = _inputs(41, [900, 1500], 12, 2, d, 4)
    g = [R.to_gpu(q, "bf16"), R.to_gpu(kc), R.to_gpu(vc), R.to_gpu(table), R.to_gpu(lens)]
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(q.shape[:3], device="cuda")
    dims = _dims(bd, 2, 12, g[1], table.shape[1], split_pages=64, kernel_path=path)
    need = stall.paged_decode_workspace_size(ctypes.byref(dims), 4, 0, 0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    dims.workspace, dims.workspace_bytes = ws.data_ptr(), need
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    st = stall.paged_decode_attention(
        ctypes.byref(dims), *(t.data_ptr() for t in g), 4, 0, 0, 0.1,
        out.data_ptr(), lse.data_ptr(), stream)
    assert st == 0
    torch.cuda.synchronize()
    f = ctypes.c_int(0)
    assert stall.svp_read_device_status(stream, ctypes.byref(f)) == 0
    assert f.value & 8
    out, lse = svp.paged_decode_attention(*g, scale=0.1, kernel_path=path)
    assert svp.read_device_status() == 0
    _check(out, lse, _reference(q, kc, vc, d, float(np.float32(0.1)), lens, table, 1.0, 1.0), d)
