"""token_logprobs on the GPU against the 64-bit form of page_ref.py.  Ranks and
alternatives are equal; log probabilities are off by the roundings of (x - m)/T
(three of its size) and of the logarithm of a sum of exponentials, each of which
is off by 2^-21 of itself (2^-22 the instruction, the rest its argument's
rounding at the distances that weigh)."""
import numpy as np
import pytest

import cache_ref as R
import page_ref as G

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


def _pack(allowed):
    n, v = allowed.shape
    bits = np.zeros((n, (v + 31) // 32 * 32), np.uint8)
    bits[:, :v] = allowed
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32)


def _check(got, ref, x, temperature):
    lp, en, rank, top, which = (t.cpu().numpy() for t in got)
    assert np.array_equal(rank, ref[2])
    assert np.array_equal(which, ref[4])
    fin = np.where(np.isfinite(x), x, 0.0)
    span = (fin.max(-1) - fin.min(-1)) / temperature + 1
    tol = 2.0 ** -20 + 2.0 ** -22 * span
    for a, b, t in ((lp, ref[0], tol), (en, ref[1], tol * 2), (top, ref[3], tol[:, None])):
        assert np.array_equal(np.isnan(a), np.isnan(b))
        assert np.array_equal(np.isneginf(a), np.isneginf(b))
        ok = np.isfinite(b)
        assert (np.abs(a[ok] - b[ok]) <= np.broadcast_to(t, b.shape)[ok]).all()


def _run(svp, x, tokens, n_top, temperature=1.0, allowed=None, dtype="f32"):
    return svp.token_logprobs(
        R.to_gpu(x.astype(np.float32), None if dtype == "f32" else "bf16"),
        R.to_gpu(np.asarray(tokens, np.int32)), n_top, temperature,
        None if allowed is None else R.to_gpu(_pack(allowed)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,v,n_top,temperature,density", [
    (1, 2, 1, 1.0, 1.0), (3, 3, 5, 1.0, 1.0), (7, 33, 40, 0.5, 0.5),
    (5, 1000, 8, 2.0, 1.0), (9, 4097, 1, 0.7, 0.3), (33, 7001, 5, 1.0, 0.01),
    (4, 32000, 20, 1.0, 1.0), (700, 5000, 3, 1.0, 0.9), (3, 131071, 64, 0.3, 0.5),
    (2, 319999, 64, 1.0, 1.0), (2, 320000, 0, 1.0, 0.9), (400, 40001, 7, 1.3, 1.0),
])
def test_logprobs(svp, dtype, n, v, n_top, temperature, density):
    rng = np.random.default_rng(v + n)
    x = rng.standard_normal((n, v)).astype(np.float32) * 2
    if dtype == "bf16":
        x = R.bf16(x)
    x = x.astype(np.float64)
    allowed = rng.random((n, v)) < density if density < 1 else None
    tokens = rng.integers(0, v, n)
    if allowed is not None:
        allowed[:, 1] = True
        tokens = np.where(rng.random(n) < 0.7, [rng.choice(np.nonzero(a)[0]) for a in allowed],
                          tokens)
    tokens = np.where(rng.random(n) < 0.2, -1, tokens)
    got = _run(svp, x, tokens, n_top, temperature, allowed, dtype)
    assert svp.read_device_status() == 0 and svp.last_launch_count() == 1
    ref = G.logprobs(x, tokens, n_top, float(np.float32(temperature)), allowed)
    _check(got, ref, x, temperature)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("v", [100, 600, 5003, 50000])
def test_many_equal_logits(svp, dtype, v):
    """Rows of one value, of two, and with half of them at the top."""
    rng = np.random.default_rng(v)
    x = np.zeros((6, v))
    x[1] = rng.integers(0, 2, v)
    x[2] = np.where(rng.random(v) < 0.5, 3.0, rng.standard_normal(v))
    x[3, v // 2:] = 1.0
    x[4] = -np.arange(v) // 700
    x[5, ::2] = -0.0                      # equal to 0
    x = R.bf16(x)
    for n_top in (1, 13, 64):
        tokens = rng.integers(0, v, 6)
        got = _run(svp, x, tokens, n_top, 1.0, None, dtype)
        _check(got, G.logprobs(x, tokens, n_top), x, 1.0)


def test_alternatives_gathered_in_one_place(svp):
    """The largest logits next to one another, and in one thread's part."""
    rng = np.random.default_rng(3)
    for v in (2000, 40000, 300001):
        x = rng.standard_normal((3, v))
        x[0, v - 70:] += 100
        x[1, :70] += 100
        x[2, np.arange(64) * (v // 64)] += 100
        x = x.astype(np.float32).astype(np.float64)
        got = _run(svp, x, [5, 6, 7], 64)
        _check(got, G.logprobs(x, [5, 6, 7], 64), x, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_off_16_byte_boundaries(svp, dtype):
    """Logits that start anywhere in memory, right at the tensor's end."""
    import torch
    rng = np.random.default_rng(4)
    for v, n in ((5, 4), (33, 3), (4099, 2), (20001, 3)):
        for shift in range(8):
            x = R.bf16(rng.standard_normal((n, v)))
            flat = torch.full((shift + n * v,), float("nan"),
                              dtype=torch.float32 if dtype == "f32" else torch.bfloat16,
                              device="cuda")
            flat[shift:] = R.to_gpu(x.astype(np.float32)).flatten().to(flat.dtype)
            allowed = rng.random((n, v)) < 0.8
            allowed[:, 0] = True
            tokens = rng.integers(0, v, n).astype(np.int32)
            got = svp.token_logprobs(flat[shift:].view(n, v), R.to_gpu(tokens), 4, 1.0,
                                     R.to_gpu(_pack(allowed)))
            _check(got, G.logprobs(x, tokens, 4, 1.0, allowed), x, 1.0)


def test_infinities_nan_and_nothing_allowed(svp):
    rng = np.random.default_rng(5)
    v = 3000
    x = rng.standard_normal((9, v))
    allowed = np.ones((9, v), bool)
    x[0, 5] = -np.inf                      # the token itself: probability 0
    x[1] = -np.inf                         # nothing
    allowed[2] = False                     # nothing
    x[3, 700] = np.nan
    x[4, 9] = np.inf
    allowed[5, 3] = False                  # the token is not allowed
    x[6, 100] = np.nan                     # a NaN that is masked
    allowed[6, 100] = False
    x[7, :] = -np.inf
    x[7, 17] = 2.0                         # one token has it all
    x[8, 800] = np.inf
    allowed[8, 800] = False
    tokens = [5, 5, 5, 5, 5, 3, 5, 17, 5]
    x = x.astype(np.float32).astype(np.float64)
    got = _run(svp, x, tokens, 4, 1.0, allowed)
    ref = G.logprobs(x, tokens, 4, 1.0, allowed)
    _check(got, ref, x, 1.0)
    lp, en = got[0].tolist(), got[1].tolist()
    assert lp[0] == lp[1] == lp[2] == lp[5] == -np.inf and en[1] == en[2] == 0
    assert np.isnan(lp[3]) and np.isnan(lp[4]) and lp[7] == 0 and en[7] == 0
    assert got[4][3, 0] == 700 and got[4][4, 0] == 9


def test_tiny_and_huge_temperatures(svp):
    rng = np.random.default_rng(6)
    x = rng.standard_normal((4, 500)).astype(np.float32).astype(np.float64)
    best = x.argmax(-1)
    for t in (1e-38, 1e-45, 1e-6):
        got = _run(svp, x, best, 3, t)
        assert (got[0] == 0).all() and (got[1].abs() < 1e-6).all()
        assert got[4][:, 0].tolist() == best.tolist() and (got[3][:, 1] < -100).all()
    got = _run(svp, x, best, 3, 1e30)
    assert (got[0] + np.log(500)).abs().max() < 1e-6
    assert (got[1] - np.log(500)).abs().max() < 1e-6


def test_large_logits(svp):
    x = np.array([[3e38, -3e38, 1e38], [1e30, 1e30, 0.0], [-3e38, -3e38, -3e38]])
    got = _run(svp, x.astype(np.float32).astype(np.float64), [0, 1, 2], 3)
    lp = got[0].tolist()
    assert lp[0] == 0 and abs(lp[1] + np.log(2)) < 1e-6 and abs(lp[2] + np.log(3)) < 1e-6
    assert got[4].tolist() == [[0, 2, 1], [0, 1, 2], [0, 1, 2]]


def test_padding_and_bad_tokens(svp):
    x = np.random.default_rng(7).standard_normal((4, 50))
    got = _run(svp, x, [-1, 50, -2 ** 31, 2 ** 31 - 1], 2)
    assert svp.read_device_status() == 4
    for t, want in zip(got, (0, 0, -1, -np.inf, -1)):
        assert (t == want).all()


def test_shapes_streams_and_refusals(svp):
    import torch
    x = torch.randn((3, 5, 777), device="cuda")
    tok = torch.randint(0, 777, (3, 5), dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mine = torch.empty((3, 5), device="cuda")
    got = svp.token_logprobs(x, tok, 4, logprobs=mine, stream=s)
    s.synchronize()
    assert got[0].data_ptr() == mine.data_ptr()
    assert [tuple(t.shape) for t in got] == [(3, 5)] * 3 + [(3, 5, 4)] * 2
    ref = G.logprobs(x.double().cpu().numpy().reshape(15, -1), tok.cpu().numpy().ravel(), 4)
    _check([t.flatten(0, 1) for t in got], ref, x.cpu().numpy().reshape(15, -1), 1.0)
    one = svp.token_logprobs(x[0, 0], tok[0, 0], 1)
    assert one[0].shape == () and torch.equal(one[0], got[0][0, 0])
    none = svp.token_logprobs(x[:0], tok[:0], 2)
    assert none[3].shape == (0, 5, 2)
    for bad in (dict(logits=x.half()), dict(logits=x.transpose(0, 1)), dict(tokens=tok.long()),
                dict(tokens=tok[0]), dict(allowed=torch.ones_like(x)), dict(n_top=-1),
                dict(allowed=torch.zeros((3, 5, 24), dtype=torch.int32, device="cuda")),
                dict(entropy=mine[0]), dict(logits=x.cpu())):
        with pytest.raises(ValueError):
            svp.token_logprobs(**{**dict(logits=x, tokens=tok), **bad})
    for bad in (dict(n_top=65), dict(temperature=0.0), dict(temperature=float("nan"))):
        with pytest.raises(svp.SvpError):
            svp.token_logprobs(x, tok, **bad)


def test_captured(svp):
    import torch
    x = torch.randn((6, 9001), device="cuda")
    tok = torch.randint(0, 9001, (6,), dtype=torch.int32, device="cuda")
    svp.token_logprobs(x, tok, 5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = svp.token_logprobs(x, tok, 5)
    for _ in range(3):
        x.normal_()
        tok.random_(0, 9001)
        graph.replay()
        for a, b in zip(held, svp.token_logprobs(x, tok, 5)):
            assert torch.equal(a, b)


# ------------------------------------------------- the calls as one step

@pytest.mark.parametrize("captured", [False, True])
def test_a_speculative_step_over_selected_pages(svp, captured):
    """Pages for the drafts, packed append, bounds, scores, selection, sparse
    attention, acceptance, log probabilities of what was emitted, and the
    rejected drafts' pages back; as single calls and as one graph."""
    import torch
    rng = np.random.default_rng(17)
    B, K, hkv, group, d, V, width = 5, 4, 2, 4, 128, 3001, 24
    T, n_select = K + 1, 7
    start = np.array([60, 200, 17, 330, 128], np.int32)
    g = torch.Generator(device="cuda").manual_seed(2)

    def rand(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    z = dict(dtype=torch.int32, device="cuda")
    table = torch.full((B, width), -1, **z)
    lens, target = torch.zeros(B, **z), R.to_gpu(start)
    free, count = R.to_gpu(rng.permutation(120).astype(np.int32)), torch.full((1,), 120, **z)
    kc, vc = (torch.full((120, hkv, 16, d), float("nan"), device="cuda",
                         dtype=torch.bfloat16) for _ in "kv")
    bnd = torch.zeros((120, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    # the prompts
    n = int(start.sum())
    slots, _ = svp.kv_assign_pages(table, lens, target, free, count, n_slots=n)
    svp.kv_append(rand(n, hkv, d).bfloat16(), rand(n, hkv, d).bfloat16(), kc, vc, slots=slots)
    svp.kv_page_bounds(kc, table, lens, bnd)
    k_new, v_new = rand(B * T, hkv, d).bfloat16(), rand(B * T, hkv, d).bfloat16()
    q = rand(B, T, hkv * group, d).bfloat16()
    tl, dl = rand(B, T, V), rand(B, K, V)
    dl.copy_(tl[:, :K] + 0.3 * dl)
    drafts = dl.argmax(-1).int()
    u = torch.rand((B, T), device="cuda", generator=g)

    def step():
        target.copy_(lens + T)
        slots, _ = svp.kv_assign_pages(table, lens, target, free, count, n_slots=B * T)
        svp.kv_append(k_new, v_new, kc, vc, slots=slots)
        svp.kv_page_bounds(kc, table, lens, bnd, n_new=T)
        s = svp.paged_page_scores(q, bnd, table, lens)
        pages = svp.paged_select_pages(s, lens, n_select, 1, (T + 30) // 16)
        out, lse = svp.paged_sparse_attention(q, kc, vc, table, lens, pages)
        tokens, accepted = svp.spec_accept(tl, dl, drafts, u)
        logs = svp.token_logprobs(tl, tokens, n_top=3)
        used = (table.clone(), lens.clone())
        target.copy_(lens - K + accepted)
        svp.kv_assign_pages(table, lens, target, free, count)
        return (s, pages, out, lse, tokens, accepted) + logs + used

    if captured:
        # nothing runs while a graph is captured: the state is where it was
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
    for _ in range(4):
        q.copy_(rand(*q.shape))
        u.copy_(torch.rand(u.shape, device="cuda", generator=g))
        before = lens.clone()
        if captured:
            graph.replay()
            s, pages, out, lse, tokens, accepted, *rest = [x.clone() for x in held]
        else:
            s, pages, out, lse, tokens, accepted, *rest = step()
        assert svp.read_device_status() == 0
        used_table, used_lens = (x.cpu().numpy() for x in rest[-2:])
        assert (rest[-1] == before + T).all()
        assert (lens == before + 1 + accepted).all()
        # every page is in a table or on the stack, once
        ids = torch.cat([table[table >= 0], free[:int(count)]])
        assert ids.sort().values.tolist() == list(range(120))
        live = [x.float().double().cpu().numpy() for x in (q, kc, vc)]
        assert np.array_equal(pages.cpu().numpy(),
                              G.select(s.cpu().numpy(), used_lens, n_select, 1, 2))
        want, wlse, _, vmax = G.sparse_attention(*live, d ** -0.5, used_lens, used_table,
                                                 pages.cpu().numpy())
        tol = 2.0 ** -8 * (vmax[..., None] + np.abs(want)) + 1e-3
        assert (np.abs(out.float().double().cpu().numpy() - want) <= tol).all()
        assert np.abs(lse.double().cpu().numpy() - wlse).max() < 1e-4
        # a page that was left out holds no product above its score
        for b in range(B):
            for h in range(hkv):
                kk = R.logical(live[1], used_table[b], h, int(used_lens[b]))
                x = np.einsum("thd,nd->thn", live[0][b, :, h * group:(h + 1) * group], kk)
                most = x.max((0, 1)) * d ** -0.5
                at = s[b, h].double().cpu().numpy()[np.arange(len(kk)) // 16]
                assert (most <= at + 1e-4).all()
        ref = G.logprobs(tl.double().cpu().numpy().reshape(-1, V),
                         tokens.cpu().numpy().ravel(), 3)
        _check([x.flatten(0, 1) for x in rest[:5]], ref,
               tl.cpu().numpy().reshape(-1, V), 1.0)
