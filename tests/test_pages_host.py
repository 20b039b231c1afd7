"""What the calls on selected pages, page assignment, packed appends and token
log probabilities refuse on the host, before any launch (no GPU), and their
plain forms checked against simpler statements."""
import ctypes

import numpy as np
import pytest

import page_ref as G

P = ctypes.c_void_p(0x1000)  # never dereferenced: every call fails its checks
ODD = ctypes.c_void_p(0x1008)
OFF = ctypes.c_void_p(0x1002)


@pytest.fixture(scope="module")
def lib():
    from spec_verify_paged_gb300 import binding, build
    build.build()
    return binding.load_library()


def _dims(**kw):
    from spec_verify_paged_gb300.binding import SvpDims
    d = SvpDims()
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
                block_size=16, max_blocks_per_seq=4, num_blocks=8, dtype=1,
                k_scale=1.0, v_scale=1.0)
    base.update(kw)
    for k, v in base.items():
        setattr(d, k, v)
    return ctypes.byref(d)


def test_bounds_arguments(lib):
    def call(d, n=1, ptrs=(P, P, P), out=P):
        return lib.kv_page_bounds(d, *ptrs, n, out, None)
    assert call(None) == -1
    assert call(_dims(), n=-1) == -1
    assert call(_dims(), n=0) == 0
    assert call(_dims(batch=0), ptrs=(None,) * 3, out=None) == 0
    assert call(_dims(max_blocks_per_seq=0), ptrs=(None,) * 3, out=None) == 0
    for i in range(3):
        assert call(_dims(), ptrs=[None if j == i else P for j in range(3)]) == -1
    assert call(_dims(), out=None) == -1
    assert call(_dims(), ptrs=(ODD, P, P)) == -1
    assert call(_dims(), out=ODD) == -1
    assert call(_dims(num_blocks=0)) == -1
    assert call(_dims(dtype=2, k_scale=0.0)) == -1
    assert call(_dims(head_dim=96)) == -2
    assert call(_dims(block_size=32)) == -2
    assert call(_dims(batch=65536)) == -2
    assert call(_dims(max_blocks_per_seq=2 ** 27, num_kv_heads=16, num_q_heads=16),
                n=2 ** 31 - 1) == -2
    assert lib.svp_last_launch_count() == 0


def test_score_arguments(lib):
    def call(d, q_len=1, scale=0.1, ptrs=(P, P, P, P), out=P):
        return lib.paged_page_scores(d, *ptrs, q_len, scale, out, None)
    assert call(None) == -1
    assert call(_dims(), q_len=0) == -1
    assert call(_dims(), q_len=17) == -2
    assert call(_dims(), scale=float("nan")) == -1
    assert call(_dims(), scale=float("inf")) == -1
    assert call(_dims(num_q_heads=6, num_kv_heads=4)) == -1
    for i in range(4):
        assert call(_dims(), ptrs=[None if j == i else P for j in range(4)]) == -1
    assert call(_dims(), out=None) == -1
    assert call(_dims(), out=OFF) == -1
    assert call(_dims(), ptrs=(ODD, P, P, P)) == -1
    assert call(_dims(), ptrs=(P, ODD, P, P)) == -1
    assert call(_dims(batch=0), ptrs=(None,) * 4, out=None) == 0
    assert lib.svp_last_launch_count() == 0


def test_select_arguments(lib):
    def call(batch=2, heads=2, blocks=4, n=4, sink=1, recent=1, ptrs=(P, P), out=P):
        return lib.paged_select_pages(batch, heads, blocks, *ptrs, n, sink, recent,
                                      out, None)
    for bad in (dict(batch=-1), dict(heads=0), dict(blocks=-1), dict(n=0),
                dict(sink=-1), dict(recent=-1), dict(sink=3, recent=2),
                dict(sink=2 ** 31 - 1, recent=2), dict(ptrs=(None, P)),
                dict(ptrs=(P, None)), dict(out=None), dict(out=OFF), dict(ptrs=(OFF, P))):
        assert call(**bad) == -1, bad
    assert call(batch=65536) == -2
    assert call(blocks=2 ** 26 + 1) == -2
    assert call(n=2 ** 26 + 1) == -2
    assert call(batch=0, ptrs=(None, None), out=None) == 0
    assert lib.svp_last_launch_count() == 0


def test_sparse_attention_arguments(lib):
    def call(d, q_len=1, n=4, tree=None, scale=0.1, ptrs=(P,) * 5, pages=P,
             out=(P, P)):
        return lib.paged_sparse_attention(d, *ptrs, q_len, pages, n, tree, scale,
                                          *out, None)
    assert call(None) == -1
    for bad in (dict(q_len=0), dict(n=0), dict(n=-1), dict(scale=float("nan")),
                dict(pages=None), dict(pages=OFF), dict(tree=OFF), dict(out=(P, None)),
                dict(out=(None, P)), dict(out=(ODD, P)), dict(out=(P, OFF)),
                dict(ptrs=(ODD, P, P, P, P)), dict(ptrs=(P, ODD, P, P, P)),
                dict(ptrs=(P, P, ODD, P, P)), dict(ptrs=(P, P, P, None, P)),
                dict(ptrs=(P, P, P, P, None))):
        assert call(_dims(), **bad) == -1, bad
    assert call(_dims(), q_len=17) == -2
    assert call(_dims(head_dim=80)) == -2
    for path in (1, 2, 3):
        assert call(_dims(kernel_path=path)) == -2
    assert call(_dims(), n=2 ** 26 + 1) == -2
    assert call(_dims(dtype=3, v_scale=0.0)) == -1
    assert call(_dims(split_pages=-1)) == -1
    assert call(_dims(max_blocks_per_seq=0)) == -1
    assert call(_dims(batch=0), ptrs=(None,) * 5, pages=None, out=(None, None)) == 0
    assert lib.svp_last_launch_count() == 0


def test_assign_arguments(lib):
    def call(batch=2, blocks=4, nb=8, ptrs=(P,) * 5, cap=8, slots=P, n=4, off=P):
        return lib.kv_assign_pages(batch, blocks, nb, *ptrs, cap, slots, n, off, None)
    for bad in (dict(batch=-1), dict(blocks=-1), dict(nb=-1), dict(cap=-1), dict(n=-1),
                dict(slots=None), dict(slots=ctypes.c_void_p(0x1004)), dict(off=OFF),
                dict(ptrs=(OFF, P, P, P, P))):
        assert call(**bad) == -1, bad
    for i in range(5):
        assert call(ptrs=[None if j == i else P for j in range(5)]) == -1
    assert call(batch=65536) == -2
    assert call(batch=0, n=0, slots=None, off=None, ptrs=(None,) * 5) == 0
    assert lib.svp_last_launch_count() == 0


def test_append_slots_arguments(lib):
    def call(d, n=1, ptrs=(P,) * 5):
        return lib.kv_append_slots(d, *ptrs, n, None)
    assert call(None) == -1
    assert call(_dims(), n=-1) == -1
    assert call(_dims(), n=0, ptrs=(None,) * 5) == 0
    for i in range(5):
        assert call(_dims(), ptrs=[None if j == i else P for j in range(5)]) == -1
    for i in range(4):
        assert call(_dims(), ptrs=[ODD if j == i else P for j in range(5)]) == -1
    assert call(_dims(), ptrs=(P, P, P, P, ctypes.c_void_p(0x1004))) == -1
    assert call(_dims(num_blocks=0)) == -1
    assert call(_dims(head_dim=32)) == -2
    assert call(_dims(dtype=3, k_scale=-1.0)) == -1
    assert lib.svp_last_launch_count() == 0


def test_logprob_arguments(lib):
    def call(rows=2, vocab=100, dtype=0, logits=P, tokens=P, n=3, t=1.0, allowed=None,
             out=(P,) * 5):
        return lib.token_logprobs(rows, vocab, dtype, logits, tokens, n, t, allowed,
                                  *out, None)
    for bad in (dict(rows=-1), dict(vocab=1), dict(dtype=2), dict(n=-1), dict(t=0.0),
                dict(t=-1.0), dict(t=float("nan")), dict(t=float("inf")),
                dict(logits=None), dict(tokens=None), dict(out=(None, P, P, P, P)),
                dict(out=(P, P, P, None, P)), dict(out=(P, P, P, P, None)),
                dict(logits=OFF), dict(dtype=1, logits=ctypes.c_void_p(0x1001)),
                dict(allowed=OFF), dict(out=(P, OFF, P, P, P))):
        assert call(**bad) == -1, bad
    assert call(vocab=320001) == -2
    assert call(n=65) == -2
    assert call(rows=2 ** 27 + 1) == -2
    assert call(rows=0, logits=None, tokens=None, out=(None,) * 5) == 0
    assert lib.svp_last_launch_count() == 0


def test_python_refusals():
    """Host tensors, shapes and types are refused by the binding."""
    torch = pytest.importorskip("torch")
    import spec_verify_paged_gb300 as svp
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    t = torch.zeros((1, 4), dtype=torch.int32)
    n = torch.ones(1, dtype=torch.int32)
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    b = torch.zeros((4, 2, 2, 64), dtype=torch.bfloat16)
    s = torch.zeros((1, 2, 4))
    i64 = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: svp.kv_page_bounds(k, t, n, b),
                 lambda: svp.paged_page_scores(q, b, t, n),
                 lambda: svp.paged_select_pages(s, n, 2),
                 lambda: svp.paged_select_pages(s, n, 0),
                 lambda: svp.paged_sparse_attention(q, k, k, t, n, s.int()),
                 lambda: svp.kv_assign_pages(t, n, n, n, n),
                 lambda: svp.kv_append(q[0], q[0], k, k, slots=i64[:1]),
                 lambda: svp.kv_append(q, q, k, k, t, n, slots=i64),
                 lambda: svp.kv_append(q, q, k, k),
                 lambda: svp.token_logprobs(s, t),
                 lambda: svp.token_logprobs(s[0], n, n_top=-1)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        svp.token_logprobs(s.double(), torch.zeros((1, 2), dtype=torch.int32))


# ------------------------------------------- the plain forms check themselves

def test_reference_bounds_are_bounds():
    rng = np.random.default_rng(1)
    x = rng.standard_normal(4000) * np.exp(rng.standard_normal(4000) * 20)
    lo, hi = G.bf16_outward(x, False), G.bf16_outward(x, True)
    assert (lo <= x).all() and (x <= hi).all()
    # neighbours in bf16 at most: one step of 2^-7 relative
    assert (hi - lo <= np.abs(x) * 2.0 ** -7).all()
    for v in (lo, hi):
        assert (v.astype(np.float32).view(np.uint32) & 0xFFFF == 0).all()


def test_reference_scores_bound_the_products():
    rng = np.random.default_rng(2)
    lens = np.array([37, 16])
    table = np.array([[3, 1, 0], [2, -1, -1]])
    k = rng.standard_normal((4, 2, 16, 64))
    b = G.bounds(k, lens, table, 100, np.zeros((4, 2, 2, 64)))
    q = rng.standard_normal((2, 3, 4, 64))
    for scale in (0.3, -0.3, 0.0):
        s, _ = G.scores(q, b, lens, table, scale)
        for i in range(2):
            for j in range(int(lens[i])):
                x = np.einsum("qhd,hd->qh", q[i].reshape(3, 4, 64)[:, :, :],
                              np.repeat(k[table[i, j // 16], :, j % 16], 2, 0)) * scale
                assert (x.reshape(3, 2, 2).max((0, 2)) <= s[i, :, j // 16] + 1e-12).all()
        assert np.isneginf(s[1, :, 1:]).all()


def test_reference_select():
    s = np.array([[[1.0, 5.0, np.nan, 5.0, 2.0, np.inf, 9.0, 0.0]]])
    assert G.select(s, [128], 4, 0, 0).tolist() == [[[1, 2, 5, 6]]]
    assert G.select(s, [128], 5, 1, 1).tolist() == [[[0, 2, 5, 6, 7]]]
    assert G.select(s, [128], 6, 1, 1).tolist() == [[[0, 1, 2, 5, 6, 7]]]
    assert G.select(s, [33], 4, 1, 1).tolist() == [[[0, 1, 2, -1]]]
    assert G.select(s, [0], 2, 1, 1).tolist() == [[[-1, -1]]]


def test_reference_sparse_is_dense_over_all_pages():
    import cache_ref as R
    rng = np.random.default_rng(3)
    lens = np.array([45, 20], np.int32)
    table, total, _ = R.pages(rng, lens)
    k, v = (rng.standard_normal((total, 2, 16, 64)) for _ in range(2))
    q = rng.standard_normal((2, 3, 4, 64))
    full = np.array([[[2, 0, 1]] * 2, [[0, -1, 1]] * 2])
    a = G.sparse_attention(q, k, v, 0.2, lens, table, full)
    b = R.attention(q, k, v, 0.2, lens, table)
    for x, y in zip(a, b):
        assert np.abs(x - y).max() < 1e-12


def test_reference_assign():
    table = np.array([[5, 6, -1], [7, -1, -1], [-1, -1, -1]], np.int32)
    lens = np.array([20, 3, 0], np.int32)
    stack = np.array([1, 2, 3, 0, 0, 0], np.int32)
    new = np.array([10, 17, 18], np.int32)
    t, n, s, c, slots, off, short = G.assign(table, lens, new, stack, 3, 40)
    # page 6 comes back, then 6, 3 and 2 are taken
    assert t.tolist() == [[5, -1, -1], [7, 6, -1], [3, 2, -1]]
    assert n.tolist() == new.tolist() and c == 1 and not short
    assert slots[:15] == list(range(115, 128)) + [96, 48] and slots[32:] == [-1] * 8
    assert off == [0, 0, 14, 32]
    t, n, _, c, slots, off, short = G.assign(table, lens, new, stack, 1, 40)
    assert n.tolist() == [10, 17, 0] and short and c == 1 and slots[14:] == [-1] * 26


def test_reference_logprobs():
    x = np.array([[0.0, 1.0, 1.0, -np.inf]])
    lp, en, rank, top, which = G.logprobs(x, [2], 4)
    z = np.log(1 + 2 * np.e)
    assert abs(lp[0] - (1 - z)) < 1e-12 and rank[0] == 1
    assert which.tolist() == [[1, 2, 0, -1]] and np.isneginf(top[0, 3])
    p = np.exp([0 - z, 1 - z, 1 - z])
    assert abs(en[0] + (p * np.log(p)).sum()) < 1e-12
    assert G.logprobs(x, [3], 0)[0][0] == -np.inf and G.logprobs(x, [3], 0)[2][0] == -1
