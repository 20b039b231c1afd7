"""What the 4-bit cache, gather, score and eviction entry points refuse, on
the host, before any launch (no GPU)."""
import ctypes

import numpy as np
import pytest

import cache_ref as R

P = ctypes.c_void_p(0x1000)  # never dereferenced: every call fails its checks


@pytest.fixture(scope="module")
def lib():
    from spec_verify_paged_gb300 import binding, build
    build.build()
    return binding.load_library()


def _dims(**kw):
    from spec_verify_paged_gb300.binding import SvpDims
    d = SvpDims()
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
                block_size=16, max_blocks_per_seq=4, num_blocks=8, dtype=3,
                k_scale=1.0, v_scale=1.0)
    base.update(kw)
    for k, v in base.items():
        setattr(d, k, v)
    return d


def test_fp4_scales_and_paths(lib):
    for kw in (dict(k_scale=0.0), dict(v_scale=-1.0), dict(k_scale=float("nan")),
               dict(v_scale=float("inf"))):
        d = _dims(**kw)
        assert lib.kv_append(ctypes.byref(d), P, P, P, P, P, P, 1, None) == -1
        assert lib.paged_decode_workspace_size(ctypes.byref(d), 1, 0, 0) == 0
    for path, d in ((1, 128), (1, 64), (3, 64)):
        d = _dims(kernel_path=path, head_dim=d)
        assert lib.paged_decode_attention(ctypes.byref(d), P, P, P, P, P, 1, 0, 0,
                                          0.1, P, P, None) in (-2, -3)
        assert lib.paged_decode_workspace_size(ctypes.byref(d), 1, 0, 0) == 0
    assert lib.paged_decode_workspace_size(ctypes.byref(_dims()), 1, 0, 0) > 0
    assert lib.paged_decode_attention(ctypes.byref(_dims(head_dim=96)), P, P, P, P,
                                      P, 1, 0, 0, 0.1, P, P, None) == -2
    assert lib.svp_last_launch_count() == 0


@pytest.mark.parametrize("which", range(4))
def test_append_fp4_alignment(lib, which):
    ptrs = [P] * 4
    ptrs[which] = ctypes.c_void_p(P.value + 8)
    assert lib.kv_append(ctypes.byref(_dims()), *ptrs, P, P, 1, None) == -1


def test_gather_arguments(lib):
    def call(d, ptrs=(P, P, P, P, None), n=1, out=(P, P)):
        return lib.kv_gather(None if d is None else ctypes.byref(d), *ptrs, n, *out, None)
    assert call(None) == -1
    assert call(_dims(), n=-1) == -1
    assert call(_dims(), n=0) == 0
    assert call(_dims(batch=0), ptrs=(None,) * 5, out=(None, None)) == 0
    assert call(_dims(), ptrs=(None, P, P, P, None)) == -1
    assert call(_dims(), out=(P, None)) == -1
    assert call(_dims(), out=(ctypes.c_void_p(P.value + 2), P)) == -1
    assert call(_dims(head_dim=80)) == -2
    assert call(_dims(block_size=32)) == -2
    assert lib.svp_last_launch_count() == 0


def test_score_arguments(lib):
    def call(d, q_len=1, n_sink=0, window=0, tree=None, scale=0.1, fresh=0,
             ptrs=(P, P, P, P, P), scores=P):
        return lib.paged_score_update(None if d is None else ctypes.byref(d), *ptrs,
                                      q_len, n_sink, window, tree, scale, fresh,
                                      scores, None)
    assert call(None) == -1
    for bad in (dict(q_len=0), dict(n_sink=-1), dict(window=-1), dict(scale=float("nan")),
                dict(fresh=-1), dict(fresh=2), dict(scores=None),
                dict(ptrs=(P, P, None, P, P)), dict(tree=P, window=4),
                dict(tree=ctypes.c_void_p(0x1002)), dict(scores=ctypes.c_void_p(0x1002)),
                dict(ptrs=(ctypes.c_void_p(0x1008), P, P, P, P))):
        assert call(_dims(), **bad) == -1, bad
    assert call(_dims(), q_len=17) == -2
    assert call(_dims(num_q_heads=6, num_kv_heads=4)) == -1
    assert call(_dims(batch=0), ptrs=(None,) * 5, scores=None) == 0
    assert lib.svp_last_launch_count() == 0


def test_evict_arguments(lib):
    def call(d, budget=16, n_sink=0, n_recent=0, dst=None, blocks=0,
             ptrs=(P, P, P, P, P), out=(P, P)):
        return lib.kv_evict(None if d is None else ctypes.byref(d), *ptrs, budget,
                            n_sink, n_recent, dst, blocks, *out, None)
    assert call(None) == -1
    for bad in (dict(budget=0), dict(n_sink=-1), dict(n_recent=-1),
                dict(n_sink=9, n_recent=8), dict(n_sink=2 ** 31 - 1, n_recent=2),
                dict(budget=65), dict(dst=P, blocks=0), dict(dst=P, blocks=1, budget=17),
                dict(ptrs=(P, P, None, P, P)), dict(out=(P, None)), dict(out=(None, P)),
                dict(ptrs=(ctypes.c_void_p(0x1008), P, P, P, P)),
                dict(ptrs=(P, P, ctypes.c_void_p(0x1002), P, P))):
        assert call(_dims(), **bad) == -1, bad
    assert call(_dims(max_blocks_per_seq=2 ** 26 + 1)) == -2
    assert call(_dims(head_dim=32)) == -2
    assert call(_dims(batch=0), ptrs=(None,) * 5, out=(None, None)) == 0
    assert lib.svp_last_launch_count() == 0


def test_python_refusals():
    """Host tensors, shapes and types are refused by the binding."""
    torch = pytest.importorskip("torch")
    import spec_verify_paged_gb300 as svp
    kc = torch.zeros((4, 2, 16, 72), dtype=torch.uint8)
    t = torch.zeros((1, 4), dtype=torch.int32)
    n = torch.ones(1, dtype=torch.int32)
    q = torch.zeros((1, 1, 4, 128), dtype=torch.bfloat16)
    s = torch.zeros((4, 2, 16))
    with pytest.raises(ValueError):
        svp.paged_decode_attention(q, kc, kc, t, n)
    with pytest.raises(ValueError):
        svp.kv_append(q, q, kc, kc, t, n)
    with pytest.raises(ValueError):
        svp.kv_gather(kc, kc, t, n, 1)
    with pytest.raises(ValueError):
        svp.kv_evict(kc, kc, s, t, n, 8)
    with pytest.raises(ValueError):
        svp.paged_score_update(q, kc, s, t, n, s)
    assert svp.fp4_row_bytes(64) == 36 and svp.fp4_row_bytes(128) == 72


# ------------------------------------------- the plain forms check themselves

def test_reference_format():
    """The reference's rounding: the E4M3 codes are their own nearest values,
    E2M1 ties go to the even code, and a stored row is within half a step."""
    grid = R.E4M3[:127]
    assert np.array_equal(R.e4m3_code(grid), np.arange(127))
    mid = (grid[:-1] + grid[1:]) / 2
    assert (R.e4m3_code(mid) % 2 == 0).all()
    rng = np.random.default_rng(0)
    x = R.bf16(rng.standard_normal((50, 128)))
    rows = R.quantise(x, 1.0)
    v = R.values(rows, "fp4", 128)
    step = np.repeat(R.E4M3[rows[:, 64:]], 16, -1)
    # the widest E2M1 spacing is 2 (4 to 6); beyond 6 a value saturates by at
    # most the scale's own half step (2^-4 relative)
    assert (np.abs(v - x) <= step * (1 + 6 / 16)).all()
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] + [0.0] * 8)
    got = R.values(R.quantise(ties[None], 1.0), "fp4", 16)[0, :8]
    assert got.tolist() == [0, 1, 1, 2, 2, 4, 4, 6]


def test_reference_attention_agrees_with_the_oracle(oracle_mod):
    """The numpy form of attention used here and the C oracle."""
    from spec_verify_paged_gb300 import workloads as W
    cfg = W.small_config(batch=2, num_q_heads=4, num_kv_heads=2, head_dim=64,
                         q_len=3, dtype="f32", ctx_min=3, ctx_max=60, seed=5)
    wl = W.make_attention(cfg)
    o, l = oracle_mod.paged_attention(wl.q, wl.k_cache, wl.v_cache, wl.block_table,
                                      wl.seq_lens, 3, 2, 20, wl.scale)
    out, lse, _, _ = R.attention(wl.q.astype(np.float64), wl.k_cache.astype(np.float64),
                                 wl.v_cache.astype(np.float64), float(wl.scale),
                                 wl.seq_lens, wl.block_table, 2, 20)
    assert np.abs(out - o).max() < 1e-12 and np.abs(lse - l).max() < 1e-12
